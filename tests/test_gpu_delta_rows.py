"""delta_rule's value elements are held to a bound one by one: neighbours of far larger magnitude, tokens that stand out, thousands of tokens,
and the float32 of batches that go token by token."""

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


@pytest.mark.parametrize("rate", [1e-4, 0.1])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,heads", [([5000, 33], 2), ([2500] * 6, 48)])
def test_thousands_of_tokens(lens, heads, dtype, rate):
    check_rows(DeltaWorld(lens, heads=heads, heads_k=heads // 2, dtype=dtype, seed=3, rate=rate), D)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_the_same_keys_over_thousands_of_tokens(dtype):
    """Eight keys in turn: what is rounded off in one direction comes again."""
    n = 2000
    w = DeltaWorld([n], heads=2, heads_k=1, dtype=dtype, seed=4, rate=1e-4)
    w.k[:n] = w.k[:8].repeat(n // 8, 1, 1)
    check_rows(w, D)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [40, 400])
def test_tokens_that_stand_out(dtype, n):
    w = DeltaWorld([n, n], dtype=dtype, seed=5)
    w.v[20:2 * n:32] *= 2.0 ** 10
    check_rows(w, D)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,save", [([1, 1, 1], False), ([8, 5, 3], False), ([12, 10, 1], False), ([9, 4, 40], True)])
def test_token_by_token(lens, save, dtype):
    n = len(lens)
    w = DeltaWorld(lens, dtype=dtype, seed=6, slots=2 * n + sum(lens) + 1)
    if save:
        w.save = [2 * n + r for r in range(w.total)]
    check_rows(w, D)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_outputs_that_cancel(dtype):
    """Queries along which the state has next to nothing: a token's outputs go by float32's rounding, not by the output's type."""
    w = DeltaWorld([6, 6], heads=2, heads_k=2, dtype=dtype, seed=7)
    for s in range(2):
        # states of one direction, queries at right angles to it
        d = torch.nn.functional.normalize(torch.randn(2, w.dim_k, device="cuda", generator=w.g), dim=-1)
        w.pool[s] = torch.randn(2, w.dim_v, 1, device="cuda", generator=w.g) * d[:, None] * 10
        r = slice(6 * s, 6 * s + 6)
        q = w.q[r].float()
        w.q[r] = (q - (q * d).sum(-1, keepdim=True) * d).to(dtype)
    w.v *= 2.0 ** -10
    check_rows(w, D)
