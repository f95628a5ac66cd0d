"""paged_attend_shared's refusals, on the host and before the first CUDA call."""

import ctypes

import pytest

from speculative_decoding_draft_kv_gb300 import build as B
from speculative_decoding_draft_kv_gb300 import paged as P
from speculative_decoding_draft_kv_gb300 import ring as R
from tests.test_paged_abi import BAD_BATCHES, BAD_CACHES, FAKE, addr, attend, batch, cache


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P._load()


def refused(lib, args, prefix):
    assert lib.paged_attend_shared(addr(args), addr(prefix), None) == R.RING_EINVAL
    assert P.paged_last_error().startswith("paged_attend_shared: ")


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(lib, bad):
    refused(lib, attend(cache(**bad), batch()), batch())


@pytest.mark.parametrize("bad", BAD_BATCHES, ids=str)
def test_bad_batches_and_prefixes(lib, bad):
    refused(lib, attend(cache(), batch(**bad)), batch())
    refused(lib, attend(cache(), batch()), batch(**bad))
    n = ctypes.c_int64()
    for a, b in ((batch(**bad), batch()), (batch(), batch(**bad))):
        assert lib.paged_attend_shared_workspace(addr(cache()), addr(a), addr(b), 16, 32, ctypes.byref(n)) == R.RING_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(o=None), dict(o=FAKE), dict(q=FAKE + 8), dict(window=1), dict(window=-1), dict(mask=3), dict(mask=P.PAGED_TREE),
    dict(tree=FAKE), dict(dtype=P.PAGED_BF16), dict(dtype=P.PAGED_F32), dict(scale=-1.0), dict(scale=float("nan")), dict(n_head=12),
    dict(n_rows=-1), dict(q_row_stride=4100)], ids=str)
def test_bad_arguments(lib, bad):
    refused(lib, attend(cache(), batch(), **bad), batch())


def test_missing_ones(lib):
    refused(lib, attend(cache(), batch()), None)
    assert lib.paged_attend_shared(None, addr(batch()), None) == R.RING_EINVAL
    assert lib.paged_attend_shared_workspace(addr(cache()), addr(batch()), None, 16, 32, ctypes.byref(ctypes.c_int64())) == R.RING_EINVAL
    assert lib.paged_attend_shared_workspace(addr(cache()), addr(batch()), addr(batch()), 16, 32, None) == R.RING_EINVAL


def test_nothing_to_do(lib):
    a = attend(cache(), batch(n_seq=0, q_start=None, kv_len=None, pages=None), workspace=None, workspace_bytes=0)
    assert lib.paged_attend_shared(addr(a), addr(batch()), None) == R.RING_OK
    a = attend(cache(), batch(), n_rows=0, q=None, o=None, workspace=None, workspace_bytes=0)
    assert lib.paged_attend_shared(addr(a), addr(batch()), None) == R.RING_OK
