"""Keys of no length: with norms they are divided by sqrt(eps) alone, which is large, and stay zero: a token that leaves its
sequence's state to its decay, whatever else is in its chunk."""

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("eps", [1e-6, 1e-12])
@pytest.mark.parametrize("every", [4, 32])
def test_zero_keys_among_others(dtype, eps, every):
    w = DeltaWorld([400, 300, 12], dtype=dtype, seed=1, rate=1e-3)
    w.k[3:w.total:every] = 0
    w.q[5:w.total:every] = 0
    w.check(D, eps=eps)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_keys_that_are_all_zero(dtype):
    """A whole chunk of them, a sequence's last tokens, and a head without any other."""
    w = DeltaWorld([200, 70], heads_k=4, dtype=dtype, seed=2)
    w.k[32:64, 0] = 0
    w.k[180:200, 1] = 0
    w.k[:w.total, 2] = 0
    w.check(D, eps=1e-12)


def test_keys_too_short_for_their_squares():
    """bf16 has keys whose square sum is nothing in float32: they count as zero."""
    w = DeltaWorld([150], dtype=BF16, seed=3)
    w.k[2:150:7] *= 2.0 ** -90
    w.check(D, eps=1e-12)


@pytest.mark.parametrize("n", [3, 100])
def test_zero_keys_without_eps(n):
    """0 / 0: the head is NaN from there on, others stay."""
    w = DeltaWorld([n], heads_k=4, seed=4)
    out, tol, slots = w.want(eps=0.0)
    w.k[1, 1] = 0
    state, batch = w.handles(D)
    o = torch.empty_like(w.v)
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o, eps=0.0)
    assert D.delta_device_error() == 0
    S, bound = slots[1]
    for h in (0, 2, 3):
        assert ((o[:, h].double() - out[:, h]).abs() <= tol[:, h]).all()
        assert torch.linalg.matrix_norm(w.pool[1, h].double() - S[h]) <= bound[h]
    assert torch.isnan(o[1:, 1]).all() and torch.isnan(w.pool[1, 1]).all()


@pytest.mark.parametrize("short", [1.0, 2.0 ** -20])
def test_zero_keys_that_are_not_normalised(short):
    """Beside unit keys, and beside short ones that beta makes up for."""
    w = DeltaWorld([330], dtype=BF16, seed=5, rate=1e-3)
    w.k = (torch.nn.functional.normalize(w.k.float(), dim=-1) * short).to(BF16)
    w.k[4:330:5] = 0
    w.check(D, normalise=False)
