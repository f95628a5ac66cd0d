"""delta_rule's value elements are held to a bound one by one: neighbours of far larger magnitude, tokens that stand out."""

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld
from tests.delta_rows_oracle import check_rows

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
BELOW = [0, 8, 20, 12, 16, 0, 4, 20, 10, 2, 14, 18, 0, 20, 6, 1]      # powers of two, of 16 value elements


def uneven(w, turn=0):
    """Value elements far below their neighbours, in v and in the states."""
    f = torch.tensor([2.0 ** -BELOW[(i + turn) % 16] for i in range(w.dim_v)], device="cuda")
    w.v = (w.v.float() * f).to(w.dtype)
    w.pool = w.pool * f[:, None]
    return w


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dims", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens,heads", [([5, 8, 1], 4), ([300, 40, 9], 4), ([70] * 20, 16)])
def test_small_value_elements_beside_large_ones(lens, heads, dims, dtype):
    """Token by token, two warps to a group, one warp to a group."""
    check_rows(uneven(DeltaWorld(lens, heads=heads, heads_k=heads // 2, dim_k=dims[0], dim_v=dims[1], dtype=dtype, seed=1)), D)


@pytest.mark.parametrize("rate", [1e-4, 0.1])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_value_elements_over_thousands_of_tokens(dtype, rate):
    check_rows(uneven(DeltaWorld([3001, 2050], heads=2, heads_k=1, dtype=dtype, seed=2, rate=rate), 3), D)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [40, 400])
def test_tokens_that_stand_out(dtype, n):
    w = DeltaWorld([n, n], dtype=dtype, seed=5)
    w.v[20:2 * n:32] *= 2.0 ** 10
    check_rows(w, D)
