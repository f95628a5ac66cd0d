"""Copies of the paged operators' handles.  No GPU needed."""

import copy
import ctypes
import gc
import pickle

import pytest

from speculative_decoding_draft_kv_gb300 import paged as P


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_a_copied_rotation_has_a_struct_that_lives_with_it(how):
    r = P.PagedRope(64, 1e4, "interleaved", "linear", 4.0)
    turns = list(r.args.turns)
    c = how(r)
    assert c.address == ctypes.addressof(c.args)
    del r
    gc.collect()
    kept = [P.PagedRope(64, 1e6) for _ in range(50)]          # what would take a freed struct's place
    at = P.PagedRopeArgs.from_address(c.address)
    assert list(at.turns) == turns and at.rotary_dim == 64 and at.layout == P.PAGED_INTERLEAVED
    assert c.inv_freq == [1e4 ** (-2 * i / 64) / 4.0 for i in range(32)] and len(kept) == 50


def test_structs_with_pointers_are_not_copied():
    """Caches and batches: a copied struct would point at tensors that nobody holds."""
    for args in (P.PagedCacheArgs(), P.PagedBatchArgs()):
        with pytest.raises(ValueError):
            copy.deepcopy(args)
        with pytest.raises(ValueError):
            pickle.dumps(args)
