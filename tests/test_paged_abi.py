"""The paged operators' C ABI: declared, exported and bound alike, and refusing bad arguments on
the host.  No GPU needed: every refusal comes before the first CUDA call."""

import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

from speculative_decoding_draft_kv_gb300 import build as B
from speculative_decoding_draft_kv_gb300 import paged as P
from speculative_decoding_draft_kv_gb300 import ring as R

HEADER = os.path.join(B.INCLUDE, "dflash_paged.h")
FAKE = 1 << 20          # an aligned address that nothing looks behind


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P._load()


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(paged_\w+)\s*\(", text, flags=re.M)))


def test_names(lib):
    assert _declared() == sorted(P.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(P.EXPORTED) <= exported


def test_layouts_match_the_binding(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"paged_cache": P.PagedCacheArgs, "paged_batch": P.PagedBatchArgs, "paged_rope": P.PagedRopeArgs,
               "paged_norm_rope_args": P.PagedNormRopeArgs, "paged_append_args": P.PagedAppendArgs,
               "paged_gather_args": P.PagedGatherArgs, "paged_attend_args": P.PagedAttendArgs}
    lines = ["#include <stdio.h>", '#include "dflash_paged.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'    printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'    printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    names = {"PAGED_F16": 0, "PAGED_BF16": 1, "PAGED_F32": 2, "PAGED_INT8": 3, "PAGED_E4M3": 4, "PAGED_CAUSAL": 0,
             "PAGED_FULL": 1, "PAGED_TREE": 2, "PAGED_HALF": 0, "PAGED_INTERLEAVED": 1, "PAGED_ERR_WAIT": 1,
             "PAGED_ERR_PAGE": 2}
    lines += [f'    printf("const {n} %d\\n", (int){n});' for n in names] + ["    return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", B.INCLUDE, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out.splitlines()}
    for c, py in structs.items():
        assert got[(c, "size")] == ctypes.sizeof(py), c
        for f, _ in py._fields_:
            assert got[(c, f)] == getattr(py, f).offset, (c, f)
    for n, v in names.items():
        assert got[("const", n)] == v == getattr(P, n)


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_stride=8 * 16 * 128, head_stride=16 * 128, row_stride=128,
             scale_page_stride=0, scale_head_stride=0, n_pages=10, page_size=16, n_head_kv=8, head_dim=128,
             format=P.PAGED_F16, reserved=0)
    d.update(kw)
    return P.PagedCacheArgs(**d)


def batch(**kw):
    d = dict(q_start=FAKE, kv_len=FAKE, pages=FAKE, pages_stride=4, n_seq=2, max_pages=4, max_q=8, max_kv=64)
    d.update(kw)
    return P.PagedBatchArgs(**d)


def rope(rotary_dim=128, layout=P.PAGED_HALF, freq=None, magnitude=1.0):
    """paged_rope_init's status and struct."""
    f = freq if freq is not None else [1.0] * max(1, rotary_dim // 2)
    r = P.PagedRopeArgs()
    rc = P._load().paged_rope_init(ctypes.addressof(r), (ctypes.c_double * len(f))(*f), magnitude, rotary_dim, layout)
    return rc, r


KEPT = []               # what an address was taken of lives on


def addr(x):
    KEPT.append(x)
    return ctypes.addressof(x) if x is not None else None


def refused(call, *args):
    assert call(*args) == R.RING_EINVAL
    assert P.paged_last_error() and P.paged_last_error() != "no error"


BAD_CACHES = [dict(k=None), dict(v=FAKE + 8), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(head_dim=96),
              dict(head_dim=0), dict(format=P.PAGED_F32), dict(format=9), dict(n_pages=0), dict(n_head_kv=0), dict(n_head_kv=65537),
              dict(row_stride=100), dict(head_stride=0), dict(page_stride=-2048), dict(page_stride=1 << 41),
              dict(format=P.PAGED_INT8), dict(format=P.PAGED_E4M3, k_scale=FAKE, v_scale=FAKE),
              dict(format=P.PAGED_INT8, k_scale=FAKE, v_scale=FAKE + 4, scale_page_stride=128, scale_head_stride=16),
              dict(format=P.PAGED_INT8, k_scale=FAKE, v_scale=FAKE, scale_page_stride=128, scale_head_stride=18)]
BAD_BATCHES = [dict(q_start=None), dict(kv_len=None), dict(pages=None), dict(n_seq=-1), dict(n_seq=70000),
               dict(max_q=-1), dict(max_q=(1 << 31) - 1), dict(max_kv=65), dict(max_pages=1 << 27, max_kv=0), dict(pages_stride=-1)]


def attend(c, b, **kw):
    d = dict(cache=addr(c), batch=addr(b), q=FAKE, o=2 * FAKE, q_row_stride=4096, q_head_stride=128, o_row_stride=4096,
             o_head_stride=128, tree=None, lse=None, workspace=FAKE, workspace_bytes=1 << 40, n_rows=16, scale=0.0,
             n_head=32, dtype=P.PAGED_F16, mask=P.PAGED_CAUSAL, window=0, reserved=0)
    d.update(kw)
    return P.PagedAttendArgs(**d)


def append(c, b, **kw):
    d = dict(cache=addr(c), batch=addr(b), k=FAKE, v=FAKE, q=None, q_out=None, k_row_stride=1024, k_head_stride=128,
             v_row_stride=1024, v_head_stride=128, n_rows=16, eps=1e-6, n_head_q=0, dtype=P.PAGED_F16)
    d.update(kw)
    return P.PagedAppendArgs(**d)


def gather(c, b, **kw):
    d = dict(cache=addr(c), batch=addr(b), k=FAKE, v=FAKE, k_row_stride=1024, k_head_stride=128, v_row_stride=1024,
             v_head_stride=128, n_rows=16, dtype=P.PAGED_F16, reserved=0)
    d.update(kw)
    return P.PagedGatherArgs(**d)


CALLS = {"paged_attend": attend, "paged_append": append, "paged_gather": gather}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches(lib, name, bad):
    c, b = cache(**bad), batch()
    refused(getattr(lib, name), addr(CALLS[name](c, b)), None)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batches(lib, name, bad):
    c, b = cache(), batch(**bad)
    refused(getattr(lib, name), addr(CALLS[name](c, b)), None)


@pytest.mark.parametrize("name", list(CALLS) + ["paged_norm_rope"])
def test_nothing_given(lib, name):
    refused(getattr(lib, name), None, None)
    if name in CALLS:
        c, b = cache(), batch()
        refused(getattr(lib, name), addr(CALLS[name](None, b)), None)
        refused(getattr(lib, name), addr(CALLS[name](c, None)), None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(o=FAKE + 2), dict(q_row_stride=4100), dict(o_head_stride=-128), dict(n_head=30), dict(n_head=0),
    dict(n_head=8 * 65), dict(dtype=P.PAGED_BF16), dict(dtype=P.PAGED_F32), dict(mask=3), dict(mask=P.PAGED_TREE),
    dict(tree=FAKE), dict(window=-1), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38),
    dict(n_rows=-1), dict(n_rows=1 << 31), dict(q=2 * FAKE), dict(q_row_stride=0), dict(o_head_stride=0),
])
def test_bad_attention(lib, bad):
    c, b = cache(), batch()
    refused(lib.paged_attend, addr(attend(c, b, **bad)), None)


def test_a_tree_has_at_most_64_nodes(lib):
    c, b = cache(), batch(max_q=65)
    refused(lib.paged_attend, addr(attend(c, b, mask=P.PAGED_TREE, tree=FAKE)), None)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=FAKE + 8), dict(k_row_stride=1023), dict(dtype=P.PAGED_BF16), dict(dtype=P.PAGED_F32),
    dict(eps=-1.0), dict(eps=math.nan), dict(n_head_q=32), dict(n_head_q=-1), dict(k_norm=FAKE + 4),
    dict(n_head_q=4, q=FAKE, q_out=FAKE, q_row_stride=512, q_head_stride=128, qo_row_stride=1024, qo_head_stride=128),
])
def test_bad_appends(lib, bad):
    c, b = cache(), batch()
    refused(lib.paged_append, addr(append(c, b, **bad)), None)


@pytest.mark.parametrize("bad", [dict(k=None), dict(v_head_stride=4), dict(dtype=P.PAGED_BF16), dict(dtype=P.PAGED_INT8)])
def test_bad_gathers(lib, bad):
    c, b = cache(), batch()
    refused(lib.paged_gather, addr(gather(c, b, **bad)), None)


ROPES = [dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144), dict(layout=2), dict(magnitude=math.inf),
         dict(rotary_dim=16, freq=[1.0] * 7 + [-1e-9]), dict(rotary_dim=16, freq=[math.nan] * 8)]


@pytest.mark.parametrize("bad", ROPES)
def test_bad_rotations(lib, bad):
    rc, r = rope(**bad)
    assert rc == R.RING_EINVAL and r.rotary_dim == 0       # untouched
    c, b = cache(), batch()
    refused(lib.paged_append, addr(append(c, b, rope=addr(r))), None)      # one that no init filled
    refused(lib.paged_norm_rope, addr(norm_rope(rope=addr(r))), None)
    refused(lib.paged_rope_init, None, (ctypes.c_double * 8)(), 1.0, 16, 0)
    rc, r = rope(128)
    assert rc == R.RING_OK
    refused(lib.paged_norm_rope, addr(norm_rope(head_dim=64, rope=addr(r))), None)


def test_turns_are_exact_fractions(lib):
    """inv_freq / 2 pi modulo 1 in units of 2^-64, against rational arithmetic; 1 / 2 pi to 40 digits."""
    from fractions import Fraction
    inv = Fraction("0.1591549430918953357688837633725143620345")
    freq = [1.0, 0.8659643233600653, 1e-6, 0.0, 6.283185307179586, 999999.5, 2.0 ** -60, 0.1]
    rc, r = rope(16, freq=freq)
    assert rc == R.RING_OK
    for f, t in zip(freq, r.turns):
        want = int(round(Fraction(f) * inv % 1 * 2 ** 64)) % 2 ** 64
        off = min((t - want) % 2 ** 64, (want - t) % 2 ** 64)
        assert off <= 1 + f * 2, (f, t, want)          # the low part of 1 / 2 pi is a double itself


def norm_rope(**kw):
    d = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, q_row_stride=4096, q_head_stride=128, k_row_stride=1024,
             k_head_stride=128, qo_row_stride=4096, qo_head_stride=128, ko_row_stride=1024, ko_head_stride=128,
             positions=FAKE, n_rows=5, eps=1e-6, n_head_q=32, n_head_k=8, head_dim=128, dtype=P.PAGED_F16)
    d.update(kw)
    return P.PagedNormRopeArgs(**d)


@pytest.mark.parametrize("bad", [
    dict(dtype=P.PAGED_INT8), dict(head_dim=80), dict(n_rows=-1), dict(n_head_q=-1), dict(eps=-1.0), dict(q=None),
    dict(k_out=None), dict(q_row_stride=4095), dict(k_head_stride=-128), dict(q_norm=FAKE + 4),
    dict(qo_row_stride=8192), dict(ko_head_stride=256),
])
def test_bad_norm_ropes(lib, bad):
    refused(lib.paged_norm_rope, addr(norm_rope(**bad)), None)
    _, r = rope()
    refused(lib.paged_norm_rope, addr(norm_rope(positions=None, rope=addr(r))), None)


def test_nothing_to_do_is_done(lib):
    c, b, none = cache(), batch(), batch(n_seq=0, q_start=None, kv_len=None, pages=None, max_pages=0, max_kv=0)
    for name, make in CALLS.items():
        assert getattr(lib, name)(addr(make(c, b, n_rows=0)), None) == R.RING_OK
        assert getattr(lib, name)(addr(make(c, none)), None) == R.RING_OK
        gone = {"q": None, "o": None} if name == "paged_attend" else {"k": None, "v": None}
        assert getattr(lib, name)(addr(make(c, b, n_rows=0, **gone)), None) == R.RING_OK     # as empty tensors are
    assert lib.paged_norm_rope(addr(norm_rope(n_rows=0)), None) == R.RING_OK
    assert lib.paged_norm_rope(addr(norm_rope(n_rows=0, q=None, q_out=None, k=None, k_out=None, positions=None)), None) == R.RING_OK


def test_workspace_refusals(lib):
    n = ctypes.c_int64()
    c, b = cache(), batch()
    refused(lib.paged_attend_workspace, addr(c), addr(b), 32, None)
    refused(lib.paged_attend_workspace, None, addr(b), 32, ctypes.byref(n))
    refused(lib.paged_attend_workspace, addr(c), None, 32, ctypes.byref(n))
    refused(lib.paged_attend_workspace, addr(c), addr(b), 31, ctypes.byref(n))


def test_frequencies():
    f, m = P.rope_frequencies(128, 1e6)
    assert m == 1.0 and f[0] == 1.0 and abs(f[-1] - 1e6 ** (-126 / 128)) < 1e-18
    g, m = P.rope_frequencies(128, 1e6, "linear", 4.0)
    assert m == 1.0 and all(abs(a - b / 4) < 1e-18 for a, b in zip(g, f))
    g, _ = P.rope_frequencies(128, 1e6, "ntk", 4.0)
    assert g[0] == 1.0 and abs(g[-1] * 4 / f[-1] - 1) < 1e-12
    g, m = P.rope_frequencies(128, 1e6, "yarn", 4.0, 4096)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-15
    turns = [4096 * x / (2 * math.pi) for x in f]
    for a, b, t in zip(g, f, turns):
        want = b if t >= 32 else b / 4 if t <= 1 else None
        assert b / 4 <= a <= b and (want is None or abs(a / want - 1) < 1e-12)
    for bad in (dict(rotary_dim=7, theta=1e4), dict(rotary_dim=8, theta=0.0), dict(rotary_dim=8, theta=1e4, factor=0),
                dict(rotary_dim=8, theta=1e4, scaling="none of these"), dict(rotary_dim=8, theta=1e4, scaling="yarn")):
        with pytest.raises(ValueError):
            P.rope_frequencies(**bad)
    with pytest.raises(ValueError):
        P.PagedRope(64, inv_freq=[1.0] * 31)


def test_the_package_names_the_operators_without_pytorch():
    """Importing the package and loading the library needs no PyTorch; .paged does."""
    code = ("import sys; sys.modules['torch'] = None; import speculative_decoding_draft_kv_gb300 as s; "
            "from speculative_decoding_draft_kv_gb300 import build")
    subprocess.run(["python", "-c", code], check=True, cwd=B.ROOT)
    import speculative_decoding_draft_kv_gb300 as S
    assert S.paged_attend is P.paged_attend and S.PagedCache is P.PagedCache
    with pytest.raises(AttributeError):
        S.paged_nothing
