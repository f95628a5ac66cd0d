"""An infinity or NaN in a token's rows: what is in front of it in its 32 tokens is right or NaN, never another number, and
what is in front of those is right."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld
from tests.delta_rows_oracle import want_rows

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("what", ["v", "k", "q", "beta", "decay"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [3, 20, 31, 32, 60, 75])
@pytest.mark.parametrize("heads", [4, 24])
def test_tokens_in_front(heads, at, value, what, dtype):
    n = 100
    w = DeltaWorld([n, n], heads=heads, heads_k=heads, dtype=dtype, seed=1)
    out, tol, _ = want_rows(w)
    x = getattr(w, what)
    if what in "qkv":
        x[at, 1, 5] = value
    else:
        x[at, 1] = value
    state, batch = w.handles(D)
    o = torch.empty_like(w.v)
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
    assert D.delta_device_error() == 0
    good = (o.double() - out).abs() <= tol
    first = at // 32 * 32
    assert good[:first].all() and good[n:].all() and good[:n, [0, *range(2, heads)]].all()
    assert (good | torch.isnan(o))[first:at].all()
    if what == "v":                                  # other value elements have nothing to do with it
        good[:n, 1, 5] = True
        assert good.all()
