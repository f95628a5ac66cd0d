"""Calls of delta_rule on two streams that are under way at the same time, one by chunks with its own workspace, one token by token."""

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("other", [[2, 3, 8], [60, 9]])
def test_two_calls_under_way(other):
    worlds = [DeltaWorld([300, 5, 40], seed=1), DeltaWorld(other, seed=2)]
    wants = [w.want() for w in worlds]
    jobs = [(*w.handles(D), [torch.empty_like(w.v) for _ in range(8)], torch.cuda.Stream()) for w in worlds]
    torch.cuda.synchronize()
    for i in range(8):
        for w, (state, batch, o, stream) in zip(worlds, jobs):
            D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o[i], stream=stream)
    assert D.delta_device_error() == 0
    for w, (_, _, outs, _), (out, tol, slots) in zip(worlds, jobs, wants):
        for o in outs:
            assert ((o.double() - out).abs() <= tol).all()
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
        for slot, (S, bound) in slots.items():
            assert (torch.linalg.matrix_norm(w.pool[slot].double() - S) <= bound).all()
