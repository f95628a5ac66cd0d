"""The gated delta rule's C ABI: declared, exported and bound alike, and refusing bad arguments on the
host.  No GPU needed: every refusal comes before the first CUDA call."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from speculative_decoding_draft_kv_gb300 import build as B
from speculative_decoding_draft_kv_gb300 import delta as D
from speculative_decoding_draft_kv_gb300 import ring as R

HEADER = os.path.join(B.INCLUDE, "dflash_delta.h")
FAKE = 1 << 20          # an aligned address that nothing looks behind


@pytest.fixture(scope="module")
def lib():
    B.build()
    return D._load()


def test_names(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(delta_\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(D.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(D.EXPORTED) <= {line.split()[-1] for line in out.splitlines() if line.strip()}
    import speculative_decoding_draft_kv_gb300 as pkg
    assert pkg.delta_rule is D.delta_rule and pkg.DeltaState is D.DeltaState


def test_layouts_match_the_binding(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"delta_state": D.DeltaStateArgs, "delta_batch": D.DeltaBatchArgs, "delta_rule_args": D.DeltaRuleArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "dflash_delta.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'    printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'    printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    names = {"DELTA_ERR_BATCH": 1, "DELTA_ERR_SLOT": 2, "DELTA_ERR_WAIT": 4}
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
        assert got[("const", n)] == v == getattr(D, n)


KEPT = []               # what an address was taken of lives on


def addr(x):
    KEPT.append(x)
    return ctypes.addressof(x) if x is not None else None


def state(**kw):
    d = dict(data=FAKE, slot_stride=32 * 128 * 128, head_stride=128 * 128, n_slots=10, n_head=32, dim_k=128, dim_v=128)
    d.update(kw)
    return D.DeltaStateArgs(**d)


def batch(**kw):
    d = dict(q_start=FAKE, slot_in=FAKE, slot_out=FAKE, save=None, n_seq=2, max_q=4)
    d.update(kw)
    return D.DeltaBatchArgs(**d)


def rule(s, b, **kw):
    d = dict(state=addr(s), batch=addr(b), q=FAKE, k=2 * FAKE, v=3 * FAKE, o=4 * FAKE, q_row_stride=2048, q_head_stride=128,
             k_row_stride=2048, k_head_stride=128, v_row_stride=4096, v_head_stride=128, o_row_stride=4096, o_head_stride=128,
             g=FAKE, beta=FAKE, g_row_stride=32, beta_row_stride=32, workspace=FAKE, workspace_bytes=1 << 40, n_rows=8,
             scale=0.0, eps=1e-6, n_head_k=16, dtype=0, normalise=1, reserved=0)
    d.update(kw)
    return D.DeltaRuleArgs(**d)


def refused(a):
    assert D._load().delta_rule(addr(a), None) == R.RING_EINVAL
    assert D.delta_last_error().startswith("delta_rule: ")


BAD_STATES = [dict(data=None), dict(data=FAKE + 8), dict(slot_stride=0), dict(slot_stride=-4), dict(slot_stride=6),
              dict(head_stride=2), dict(head_stride=1 << 40), dict(n_slots=0), dict(n_head=0), dict(n_head=65552), dict(dim_k=32),
              dict(dim_k=96), dict(dim_v=256), dict(dim_v=0)]
BAD_BATCHES = [dict(q_start=None), dict(slot_in=None), dict(slot_out=None), dict(n_seq=-1), dict(n_seq=65537), dict(max_q=-1),
               dict(max_q=(1 << 31) - 1)]


@pytest.mark.parametrize("bad", BAD_STATES, ids=str)
def test_bad_states(lib, bad):
    refused(rule(state(**bad), batch()))
    n = ctypes.c_int64()
    assert lib.delta_rule_workspace(addr(state(**bad)), addr(batch()), 8, 16, ctypes.byref(n)) == R.RING_EINVAL


@pytest.mark.parametrize("bad", BAD_BATCHES, ids=str)
def test_bad_batches(lib, bad):
    refused(rule(state(), batch(**bad)))
    n = ctypes.c_int64()
    assert lib.delta_rule_workspace(addr(state()), addr(batch(**bad)), 8, 16, ctypes.byref(n)) == R.RING_EINVAL


@pytest.mark.parametrize("bad", [
    dict(state=None), dict(batch=None), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=FAKE + 2), dict(o=FAKE),
    dict(o=3 * FAKE), dict(o=2 * FAKE), dict(q_row_stride=0), dict(k_head_stride=4), dict(v_row_stride=-4096),
    dict(o_head_stride=1 << 39), dict(g=None), dict(beta=None), dict(g=FAKE + 2), dict(beta=FAKE + 1), dict(g_row_stride=0),
    dict(beta_row_stride=-32), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(n_head_k=0), dict(n_head_k=5), dict(n_head_k=64), dict(dtype=2), dict(dtype=7), dict(n_rows=-1),
    dict(n_rows=1 << 31)], ids=str)
def test_bad_arguments(lib, bad):
    refused(rule(state(), batch(), **bad))


def test_nothing_to_do(lib):
    """An empty batch's pointers are not looked at, and nothing is launched."""
    a = rule(state(), batch(n_seq=0, q_start=None, slot_in=None, slot_out=None), n_rows=0, q=None, k=None, v=None, o=None, g=None,
             beta=None, workspace=None, workspace_bytes=0)
    assert lib.delta_rule(addr(a), None) == R.RING_OK
    assert lib.delta_rule(None, None) == R.RING_EINVAL
    n = ctypes.c_int64()
    assert lib.delta_rule_workspace(addr(state()), addr(batch()), 8, 16, None) == R.RING_EINVAL
    assert lib.delta_rule_workspace(addr(state()), addr(batch()), 8, 16, ctypes.byref(n)) == R.RING_OK and n.value >= 0


def test_the_binding_refuses_what_is_not_on_the_gpu():
    import torch
    with pytest.raises(TypeError):
        D.DeltaState(torch.zeros(1, 1, 64, 64))
    with pytest.raises(TypeError):
        D.DeltaBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1)
