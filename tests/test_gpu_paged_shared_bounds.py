"""paged_attend_shared where some row bounds are wrong, of beginnings or of sequences: a bound that decreases, or lies far
outside, is reported, and all those whose own bounds are right keep their rows, wherever they stand."""

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from tests.test_gpu_paged_shared import Shared

pytestmark = pytest.mark.gpu


def spans(start, rows, most):
    return [(a, b) if 0 <= a <= b <= rows and b - a <= most else None for a, b in zip(start, start[1:])]


def run(s, p_start=None, q_start=None, max_q=None, p_max_q=None):
    """The call with other bounds: (o, lse, queries, whose rows are right)."""
    w, n = s.w, len(s.own)
    cache, _, _ = s.handles()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    q_start = [int(x) for x in w.q_start[:n + 1]] if q_start is None else q_start
    p_start = [int(x) for x in s.p_start] if p_start is None else p_start
    max_q = max_q or max(a for a, _ in s.own)
    p_max_q = p_max_q or w.total
    batch = P.PagedBatch(ints(q_start), w.kv_len[:n], w.pages[:n], max_q)
    prefix = P.PagedBatch(ints(p_start), w.kv_len[n:], w.pages[n:], p_max_q)
    q = w.randn(w.heads)
    o = torch.full_like(q, 7.0)
    lse = torch.full((w.rows, w.heads), 7.0, device="cuda")
    size = P.paged_attend_shared_workspace(cache, batch, prefix, w.rows, w.heads)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")        # whatever an earlier call left there
    P.paged_attend_shared(cache, batch, prefix, q, o, lse=lse, workspace=ws)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
    return o, lse, q, spans(q_start, w.rows, max_q), spans(p_start, w.rows, p_max_q)


def check(s, **kw):
    o, lse, q, own, prefixes = run(s, **kw)
    w = s.w
    rows = [[] if x is None else list(range(*x)) for x in own]
    mine = {r: next((k for k, y in enumerate(prefixes) if y is not None and y[0] <= r < y[1]), None) for x in rows for r in x}
    left = torch.ones(w.rows, dtype=torch.bool)
    left[list(mine)] = False
    # as many times over as a sequence's rows have different beginnings
    kinds = [sorted({mine[r] for r in x}, key=str) for x in rows]
    for turn in range(max(map(len, kinds))):
        has = [x[turn] if turn < len(x) else None for x in kinds]
        want, wl, tol, ltol = s.contexts(has).attend(q)
        good = ((o.double() - want).abs() <= tol).flatten(1).all(1) & ((lse.double() - wl).abs() <= ltol).all(1)
        for j, x in enumerate(rows):
            for r in x:
                assert mine[r] != has[j] or good[r], (r, j, mine[r])
    assert (o[left.cuda()] == 7).all() and (lse[left.cuda()] == 7).all()


GROUPS = [dict(heads=4, kv_heads=2), dict(heads=32, kv_heads=1)]      # few and many query rows


@pytest.mark.parametrize("kw", GROUPS, ids=str)
@pytest.mark.parametrize("p_start", [[0, 4, -1, 8, 12], [0, 4, 1 << 30, 8, 12], [8, 12, 0, 4, 4], [0, 2, 9, 5, 5], [0, 10, 3, 3, 3]], ids=str)
def test_beginnings_beside_a_wrong_bound(p_start, kw):
    check(Shared([(4, 30), (2, 17), (4, 40), (2, 2)], [(100, 1), (33, 1), (257, 1), (64, 1)], seed=1, **kw), p_start=p_start)


@pytest.mark.parametrize("kw", GROUPS, ids=str)
@pytest.mark.parametrize("at,bad", [(2, -1), (2, 1 << 30), (1, -2 ** 31), (3, 2)])
def test_sequences_beside_a_wrong_bound(at, bad, kw):
    s = Shared([(4, 30), (4, 17), (4, 40), (4, 5), (4, 300)], [(100, 3), (33, 2)], seed=2, **kw)
    q_start = [0, 4, 8, 12, 16, 20]
    q_start[at] = bad
    check(s, q_start=q_start, max_q=5)


@pytest.mark.parametrize("n,per", [(20, 4), (70, 3), (300, 2)])
@pytest.mark.parametrize("bad", [-9, 1 << 30, 3])
def test_in_the_middle_of_many(n, per, bad):
    """More than a warp looks at at once."""
    s = Shared([(2, 5 + i % 40) for i in range(n)], [(20 + 7 * i, per) for i in range(n // per)], heads=2, kv_heads=1, dim=64, seed=3)
    q_start = [2 * i for i in range(n + 1)]
    p_start = [2 * per * i for i in range(n // per + 1)]
    q_start[n // 2] = bad
    p_start[len(p_start) // 2 + 1] = bad
    check(s, q_start=q_start, p_start=p_start, max_q=2, p_max_q=2 * per)
