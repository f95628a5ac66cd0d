"""The order of what the roles inside an attention CTA read and write: items one behind another in the
same shared memory, again and again, with the same bits each time."""

import ctypes
import subprocess

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import build as B
from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import World
from tests.test_gpu_paged_attend import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "bf16"), ("int8", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("chunk", [0, 150])
def test_dealt_items_one_behind_another(fmt, dtype, dim, chunk):
    """Verify blocks of 9 tokens, 4 heads to a kv head: 36 rows, so that of block 0's warps two have rows
    and two run straight on into the next item, whose queries' powers of two they write while the
    others still read the odd tiles' sums of this one.  With a chunk among them, in the variant of two blocks."""
    lens = [(9, 140 + (i * 173) % 900) for i in range(64)]
    if chunk:
        lens[40] = (chunk, 700)
    w = World(lens, heads=32, kv_heads=8, page=16, fmt=fmt, dtype=dtype, dim=dim, seed=dim + chunk)
    # rows' magnitudes far apart, so that a power of two of another row or item does not go unseen
    q = w.randn(w.heads) * torch.exp2(torch.randint(-3, 4, (w.rows, w.heads, 1), generator=w.g, device="cuda")).to(w.dtype)
    want = check(w, q=q)
    cache, batch = w.handles(P)
    ws = torch.empty(P.paged_attend_workspace(cache, batch, w.heads), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(w.rows, w.heads, device="cuda")
    first = None
    for _ in range(25):
        o.fill_(7.0)
        P.paged_attend(cache, batch, q, o, lse=lse, workspace=ws)
        first = lse.clone() if first is None else first
        assert torch.equal(o, want) and torch.equal(lse, first)
    assert P.paged_device_error() == 0


PROBE = r"""
#include "paged_ptx.h"
using namespace dflash;
// Four warps that meet twice a round, as the streaming kernel's do at an item's end, and a fifth that raises
// a flag after `late` clocks; the round in which each of the four left.
__global__ void probe(int late, int rounds, int *left) {
    __shared__ volatile int flag;
    if (threadIdx.x == 0) flag = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if (warp == 4) {
        const long long t0 = clock64();
        while (clock64() - t0 < late) {}
        if ((threadIdx.x & 31) == 0) flag = 1;
        return;
    }
    int i = 0;
    for (; i < rounds; ++i) {
        if (bar_any(1, 128, flag != 0)) break;
        bar_sync(1, 128);
    }
    if ((threadIdx.x & 31) == 0) left[blockIdx.x * 4 + warp] = i;
}
extern "C" int run(int late, int rounds, int blocks, int *left) {
    probe<<<blocks, 160>>>(late, rounds, left);
    return (int)cudaDeviceSynchronize();
}
"""


def test_warps_leave_a_barrier_together(tmp_path):
    """Whenever a flag is raised, all the warps that vote on it leave in the same round: none is left at the
    next barrier, which has no limit.  (The rounds are limited, so every warp leaves in the end.)"""
    src, lib = tmp_path / "probe.cu", tmp_path / "probe.so"
    src.write_text(PROBE)
    subprocess.run([B._nvcc(), *B.ARCH, *B.FLAGS, "-shared", str(src), "-o", str(lib)], check=True)
    run = ctypes.CDLL(str(lib)).run
    run.argtypes = [ctypes.c_int] * 3 + [ctypes.c_void_p]
    rounds, blocks = 2000, 64
    seen = set()
    for late in list(range(0, 4000, 37)) + [1 << 30 >> k for k in range(14, 20)]:
        left = torch.full((blocks, 4), -1, dtype=torch.int32, device="cuda")
        assert run(late, rounds, blocks, left.data_ptr()) == 0
        assert (left >= 0).all() and (left == left[:, :1]).all(), (late, left.tolist())
        seen.update(left.flatten().tolist())
    assert len(seen) > 20                        # flags raised in many different rounds
