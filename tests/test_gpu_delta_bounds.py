"""delta_rule where some row bounds are wrong: a bound that decreases, or lies far outside, is reported, and every sequence whose
own bounds are right gets its result all the same, wherever it stands in the batch."""

import copy

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld

pytestmark = pytest.mark.gpu


def alone(w, s, first, last):
    """Sequence s of rows first .. last - 1 as a world of its own."""
    x = copy.copy(w)
    for name in ("q", "k", "v", "decay", "beta"):
        setattr(x, name, getattr(w, name)[first:last])
    x.lens, x.starts, x.total, x.rows = [last - first], [0, last - first], last - first, last - first
    x.slot_in, x.slot_out = [w.slot_in[s]], [w.slot_out[s]]
    return x


def check(q_start, rows, max_q, **kw):
    n = len(q_start) - 1
    w = DeltaWorld([0] * n, spare_rows=rows, **kw)
    y = DeltaWorld([rows], **kw)
    for name in ("q", "k", "v", "decay", "beta"):
        setattr(w, name, getattr(y, name))
    spans = [(a, b) if 0 <= a <= b <= rows and b - a <= max_q else None for a, b in zip(q_start, q_start[1:])]
    wants = [None if x is None else alone(w, s, *x).want() for s, x in enumerate(spans)]
    state, batch = D.DeltaState(w.pool), D.DeltaBatch(w.ints(q_start), w.ints(w.slot_in), w.ints(w.slot_out), max_q)
    before, o = w.pool.clone(), torch.full_like(w.v, 7.0)
    # whatever an earlier call left in the workspace
    ws = torch.full((D.delta_rule_workspace(state, batch, rows, w.heads_k),), 255, dtype=torch.uint8, device="cuda")
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o, workspace=ws)
    assert D.delta_device_error() == D.DELTA_ERR_BATCH
    covered = torch.zeros(rows, dtype=torch.int32)
    for x in spans:
        if x is not None:
            covered[x[0]:x[1]] += 1
    assert covered.max() == 1, "rows of two sequences may hold anything"
    for s, (x, want) in enumerate(zip(spans, wants)):
        slot = w.slot_out[s]
        if x is None:
            assert torch.equal(w.pool[slot].view(torch.int32), before[slot].view(torch.int32)), s
            continue
        out, tol, slots = want
        off = (o[x[0]:x[1]].double() - out).abs()
        assert (off <= tol).all(), (s, x)
        S, bound = slots[slot]
        assert (torch.linalg.matrix_norm(w.pool[slot].double() - S) <= bound).all(), s
    assert (o[(covered == 0).cuda()] == 7).all()


@pytest.mark.parametrize("heads,heads_k", [(2, 1), (24, 12)])
@pytest.mark.parametrize("q_start,rows", [
    ([0, 200, -1, 600, 800], 800),                 # the first sequence's later chunks are behind a bound below them
    ([0, 200, 100_000, 600, 800], 800),            # one far above
    ([0, 1000, -5, 20], 1000),
    ([0, 300, 120, 120], 300),                     # an empty sequence that begins inside the first one
    ([500, 600, 0, 100], 600),                     # later rows first
    ([160, 200, 200, 200, 200, 0, 100], 200),      # and two sequences whose chunks would have one place
    ([-2 ** 31, 40, 2 ** 31 - 1, 40, 90], 90),
], ids=str)
def test_sequences_beside_a_wrong_bound(q_start, rows, heads, heads_k):
    check(q_start, rows, 1000, heads=heads, heads_k=heads_k, seed=len(q_start))


@pytest.mark.parametrize("n", [40, 150, 1100])
@pytest.mark.parametrize("bad", [-7, 1 << 30, 25, 900])
def test_one_of_many(n, bad):
    """In the middle of many: more than a warp looks at at once, than are put in order, than it looks at in two rounds."""
    lens = [(1, 20, 9, 35)[i % 4] if i < 60 else 1 for i in range(n)]
    q_start = [sum(lens[:i]) for i in range(n + 1)]
    rows, at = q_start[-1], min(n // 2, 45)
    q_start[at] = bad
    check(q_start, rows, 40, heads=1, heads_k=1, dim_k=64, dim_v=64, seed=n)
