"""A kernel that a device cannot be set up for fails the calls that want it, and no others: the entry points
compiled against launchers that do nothing and a set-up of the tensor-core kernels that fails."""

import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import build as B
from speculative_decoding_draft_kv_gb300 import paged as P
from speculative_decoding_draft_kv_gb300 import ring as R

pytestmark = pytest.mark.gpu

STUBS = """
#include "paged.h"
namespace dflash {
cudaError_t launch_paged_rows(const PagedRowsArgs &, int, int, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_paged_gather(const PagedGatherArgs &, int, int, cudaStream_t) { return cudaSuccess; }
#define OF(T) \\
    template <> cudaError_t paged_attend_setup_t<T>() { return cudaSuccess; } \\
    template <> cudaError_t paged_prefill_setup_t<T>() { return cudaErrorLaunchOutOfResources; } \\
    template <> cudaError_t launch_paged_attend_t<T>(const PagedAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t) { return cudaSuccess; } \\
    template <> cudaError_t launch_paged_prefill_t<T>(const PagedAttendArgs &, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t) { return cudaErrorUnknown; }
OF(PAGED_F16)
OF(PAGED_BF16)
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("stubs")
    src, out = d / "stubs.cu", d / "paged_host.so"
    src.write_text(STUBS)
    subprocess.run([B._nvcc(), *B.ARCH, *B.FLAGS, "-shared", os.path.join(B.CSRC, "paged_host.cu"), str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    for name in ("paged_norm_rope", "paged_append", "paged_gather", "paged_attend"):
        getattr(lib, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.paged_attend_workspace.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    lib.paged_last_error.restype = ctypes.c_char_p
    return lib


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_other_calls_are_served(lib, dtype):
    room = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda").data_ptr()
    fmt = P._TYPES[dtype]
    cache = P.PagedCacheArgs(room, room, None, None, 8 * 16 * 128, 16 * 128, 128, 0, 0, 4, 16, 8, 128, fmt, 0)
    batch = P.PagedBatchArgs(room, room, room, 4, 2, 4, 8, 64)
    c, b = ctypes.addressof(cache), ctypes.addressof(batch)
    rows = dict(k=room, v=room, k_row_stride=1024, k_head_stride=128, v_row_stride=1024, v_head_stride=128, n_rows=16, dtype=fmt)
    calls = {
        "paged_norm_rope": P.PagedNormRopeArgs(k=room, k_out=room, k_row_stride=1024, k_head_stride=128, ko_row_stride=1024, ko_head_stride=128,
                                               n_rows=16, eps=1e-6, n_head_k=8, head_dim=128, dtype=fmt),
        "paged_append": P.PagedAppendArgs(cache=c, batch=b, eps=1e-6, **rows),
        "paged_gather": P.PagedGatherArgs(cache=c, batch=b, **rows),
    }
    for name, args in calls.items():
        assert getattr(lib, name)(ctypes.addressof(args), None) == R.RING_OK, lib.paged_last_error()
    size = ctypes.c_int64()
    for max_q, want in ((1, R.RING_OK), (40, R.RING_ECUDA), (1, R.RING_OK), (40, R.RING_ECUDA)):
        batch.max_q = max_q
        assert lib.paged_attend_workspace(c, b, 32, ctypes.byref(size)) == R.RING_OK
        work = torch.zeros(size.value, dtype=torch.uint8, device="cuda")
        args = P.PagedAttendArgs(cache=c, batch=b, q=room, o=room + (1 << 18), q_row_stride=4096, q_head_stride=128, o_row_stride=4096,
                                 o_head_stride=128, workspace=work.data_ptr(), workspace_bytes=size.value, n_rows=16, n_head=32, dtype=fmt)
        assert lib.paged_attend(ctypes.addressof(args), None) == want, lib.paged_last_error()
        if want:
            assert b"set-up" in lib.paged_last_error()
