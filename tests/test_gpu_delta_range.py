"""delta_rule at the ends of float32's range: states that vanish within a chunk, and values near the largest there are."""

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld
from tests.delta_rows_oracle import check_rows

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("value", [0.0, 1e-30, 1e-20])
@pytest.mark.parametrize("n", [3, 64, 200])
def test_a_large_state_that_vanishes(value, n):
    """By strong decays at every token, by a single one that drops it, and little or nothing that takes its place."""
    w = DeltaWorld([n], dtype=BF16, heads=4, heads_k=2, seed=1)
    w.pool[0] *= 1e9
    w.v[:n] *= value
    w.decay[:n, 0] = -80.0
    w.decay[n // 2, 1] = -1e4
    w.decay[:n, 2] = -3.0
    check_rows(w, D)


@pytest.mark.parametrize("shift", [0, 18])
@pytest.mark.parametrize("big", [1e12, 1e25])
def test_a_state_that_comes_and_goes(big, shift):
    """Large values, a drop, small ones, a drop, large ones again: no unit of one is another's.  At the beginning of
    32 tokens and in their midst."""
    n = 300
    w = DeltaWorld([n], dtype=BF16, seed=2)
    w.pool[0] *= big
    for first, size in ((0, big), (64, 1 / big), (128, big), (160, 0.0), (224, 1 / big)):
        first += shift if first else 0
        w.decay[first] = -1e4
        w.v[first:] = w.v[first:].sign() * size
    check_rows(w, D)


@pytest.mark.parametrize("n", [5, 40, 300])
def test_values_near_the_largest(n):
    """Sums of a chunk's magnitudes pass float32 where the results do not."""
    w = DeltaWorld([n], dtype=BF16, spread=3e37, seed=3)
    check_rows(w, D)
