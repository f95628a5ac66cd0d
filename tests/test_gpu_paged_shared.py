"""paged_attend_shared against the float64 form over each row's whole context: beginnings of all lengths and
numbers, rows that have none, masks that leave rows empty, and what must not matter."""

import copy
import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import World
from tests.test_gpu_paged_attend import FORMATS, trees

pytestmark = pytest.mark.gpu


class Shared:
    """``own``: (new, own cached) of each sequence; ``prefixes``: (length, number of its sequences, in a row);
    ``skip``: sequences in front of the first that has one."""

    def __init__(self, own, prefixes, skip=0, **kw):
        self.own, self.prefixes, self.skip = own, prefixes, skip
        self.w = World(own + [(0, length) for length, _ in prefixes], **kw)
        n = len(own)
        self.first = [skip + sum(c for _, c in prefixes[:i]) for i in range(len(prefixes) + 1)]
        starts = [sum(a for a, _ in own[:i]) for i in range(n + 1)]
        self.p_start = torch.tensor([starts[i] for i in self.first], dtype=torch.int32, device="cuda")
        has = [next((i for i in range(len(prefixes)) if self.first[i] <= s < self.first[i + 1]), None) for s in range(n)]
        self.whole = self.contexts(has)

    def contexts(self, has):
        """What the rows attend to, as sequences of their own: has[s] is the number of s's beginning, or None."""
        x, n = copy.copy(self.w), len(self.own)
        x.lens, x.K, x.V = [], [], []
        for s, (a, kv) in enumerate(self.own):
            x.lens.append((a, kv + (0 if has[s] is None else self.prefixes[has[s]][0])))
            for mine, src in ((x.K, self.w.K), (x.V, self.w.V)):
                mine.append(src[s] if has[s] is None else torch.cat([src[n + has[s]], src[s]]))
        return x

    def handles(self, max_q=None, p_max_q=None):
        w, n = self.w, len(self.own)
        cache = P.PagedCache(w.k, w.v, w.ks, w.vs)
        rows = [int(x) for x in self.p_start]
        batch = P.PagedBatch(w.q_start[:n + 1], w.kv_len[:n], w.pages[:n], max_q or max(a for a, _ in self.own))
        prefix = P.PagedBatch(self.p_start, w.kv_len[n:], w.pages[n:],
                              p_max_q or max([b - a for a, b in zip(rows, rows[1:])] + [0]))
        return cache, batch, prefix

    def check(self, mask="causal", tree=None, scale=None, q=None, stride=False, errors=0, **kw):
        w = self.w
        q = w.randn(w.heads) if q is None else q
        cache, batch, prefix = self.handles(**kw)
        o = torch.full((w.rows, w.heads, w.dim), 7.0, dtype=w.dtype, device="cuda")
        if stride:
            wide = torch.full((w.rows, w.heads + 3, w.dim + 8), 7.0, dtype=w.dtype, device="cuda")
            o = wide[:, 1:1 + w.heads, :w.dim]
        ls = torch.full((w.rows, w.heads), 7.0, device="cuda")
        P.paged_attend_shared(cache, batch, prefix, q, o, mask=mask, scale=scale or 0.0, tree=tree, lse=ls)
        want, wl, tol, ltol = self.whole.attend(q, mask, 0, tree, scale, True)
        assert P.paged_device_error() == errors
        bad = ~((o[:w.total].double() - want).abs() <= tol)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                               float(((o[:w.total].double() - want).abs() / tol).max()))
        assert (o[w.total:] == 7.0).all() and (ls[w.total:] == 7.0).all(), "rows behind the batch"
        gl, none = ls[:w.total].double(), torch.isinf(wl)
        assert torch.equal(gl[none], wl[none])
        assert ((gl - wl)[~none].abs() <= ltol[~none]).all()
        return o


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("own,prefixes", [
    ([(1, 1)], [(1, 1)]), ([(1, 5), (1, 70)], [(64, 2)]), ([(1, 9)] * 12, [(333, 12)]), ([(9, 9), (3, 100), (1, 1)], [(129, 3)]),
    ([(30, 40), (64, 64), (1, 200)], [(700, 2), (65, 1)]),
])
def test_types_and_lengths(fmt, dtype, dim, own, prefixes):
    Shared(own, prefixes, fmt=fmt, dtype=dtype, dim=dim, spare_rows=2, seed=len(own) + dim).check()


@pytest.mark.parametrize("length", [1, 15, 16, 63, 64, 65, 127, 128, 129, 1000, 5000])
@pytest.mark.parametrize("n", [1, 40])
def test_lengths_of_the_beginning(length, n):
    Shared([(1, 3)] * n, [(length, n)], seed=length).check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (7, 1), (10, 2), (64, 1), (33, 3)])
@pytest.mark.parametrize("n", [1, 6, 70])
def test_head_groups(heads, kv_heads, n):
    Shared([(2, 30)] * n, [(300, n)], heads=heads, kv_heads=kv_heads, seed=heads).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fmt,order", [("f16", "hnd"), ("bf16", "nhd"), ("int8", "nhd"), ("e4m3", "hnd")])
def test_pages(page, fmt, order):
    dtype = "f16" if fmt in ("f16", "int8") else "bf16"
    Shared([(2, page + 1), (3, page - 1), (17, 3 * page)], [(2 * page + 5, 3)], page=page, fmt=fmt, dtype=dtype, order=order,
           seed=page).check()


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("e4m3", "bf16")])
def test_rows_without_a_beginning(fmt, dtype):
    """In front of the first prefix, behind the last, and with one of length 0."""
    own = [(1, 20), (3, 3), (2, 90), (5, 64), (1, 1), (2, 300)]
    Shared(own, [(100, 1), (0, 2), (257, 1)], skip=1, fmt=fmt, dtype=dtype, seed=2).check()
    Shared(own, [], fmt=fmt, dtype=dtype, seed=3).check()
    Shared(own, [(0, 6)], fmt=fmt, dtype=dtype, seed=4).check()


def test_many_prefixes_and_sequences():
    own = [(1 + i % 3, 3 + 7 * i % 90) for i in range(200)]
    Shared(own, [(1 + 37 * i % 400, 1 + i % 5) for i in range(45)], skip=3, seed=5).check()


@pytest.mark.parametrize("mask", ["full", "tree"])
@pytest.mark.parametrize("fmt,dtype", FORMATS)
def test_masks(mask, fmt, dtype):
    s = Shared([(31, 60), (64, 64), (1, 1), (9, 137)], [(200, 3), (70, 1)], fmt=fmt, dtype=dtype, spare_rows=2, seed=6)
    s.check(mask, trees(s.w) if mask == "tree" else None)


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16")])
def test_rows_that_see_nothing_of_their_own(fmt, dtype):
    """A row without tree bits and context has its beginning alone, or nothing: 0 and -inf."""
    s = Shared([(5, 5), (40, 40), (6, 6)], [(90, 2)], fmt=fmt, dtype=dtype, seed=7)
    o = s.check("tree", trees(s.w, empty=(0, 3, 7, 44, 46)))
    assert (o[46] == 0).all() and (o[0] != 0).any()


def test_a_bound_inside_a_sequence():
    """Bounds of rows, not of sequences: some tokens of a sequence have the beginning, others do not."""
    s = Shared([(4, 30), (6, 50)], [(100, 1)], seed=8)
    s.p_start = torch.tensor([2, 7], dtype=torch.int32, device="cuda")
    w = s.w
    q = w.randn(w.heads)
    cache, batch, prefix = s.handles()
    o = torch.empty_like(q)
    P.paged_attend_shared(cache, batch, prefix, q, o)
    assert P.paged_device_error() == 0
    for has, rows in ((False, [0, 1, 7, 8, 9]), (True, [2, 3, 4, 5, 6])):
        want, _, tol, _ = s.contexts([0, 0] if has else [None, None]).attend(q)
        assert ((o[rows].double() - want[rows]).abs() <= tol[rows]).all()


@pytest.mark.parametrize("far", [-1.0, 1.0])
def test_one_part_outweighs_the_other(far):
    """Scores of the beginning 60 above or below the own ones: the lighter part still counts for what it is."""
    s = Shared([(2, 40)] * 5, [(150, 5)], heads=2, kv_heads=1, seed=9)
    w = s.w
    q = w.randn(w.heads)
    q[:, :, 0] = 30.0
    for i, (_, length) in enumerate(w.lens[5:]):
        p = torch.arange(length, device="cuda")
        w.k[w.pages[5 + i][p // w.page].long(), :, p % w.page, 0] = far * 22
        w.K[5 + i][:, :, 0] = far * 22
    for j in range(5):
        s.whole.K[j] = torch.cat([w.K[5], w.K[j]])
    s.check(q=q)


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scale_and_strides(scale):
    Shared([(3, 50), (20, 60)], [(111, 2)], spare_rows=1, seed=10).check(scale=scale, stride=True)


def test_what_nobody_sees_may_hold_anything():
    s = Shared([(1, 17), (2, 40)], [(45, 2)], seed=11)
    s.w.pages[2, 3:] = 1 << 30                       # behind the beginning's last page
    s.check()


@pytest.mark.parametrize("n", [1, 12])
def test_broken_prefixes_are_reported(n):
    def run(p_start=None, p_len=None, page=None):
        s = Shared([(2, 30)] * (2 * n), [(100, n), (80, n)], seed=12)
        cache, batch, prefix = s.handles()
        lens = s.w.kv_len[2 * n:].clone()
        pages = s.w.pages[2 * n:].clone()
        if p_len is not None:
            lens[1] = p_len
        if page is not None:
            pages[1, 0] = page
        starts = s.p_start if p_start is None else torch.tensor(p_start, dtype=torch.int32, device="cuda")
        prefix = P.PagedBatch(starts, lens, pages, 2 * n)
        q = s.w.randn(s.w.heads)
        o = torch.full_like(q, 7.0)
        P.paged_attend_shared(cache, batch, prefix, q, o)
        assert P.paged_device_error() == P.PAGED_ERR_PAGE
        want, _, tol, _ = s.whole.attend(q)
        alone, _, tol1, _ = s.contexts([None] * (2 * n)).attend(q)
        good = ((o.double() - want).abs() <= tol).flatten(1).all(1)
        own = ((o.double() - alone).abs() <= tol1).flatten(1).all(1)
        return good, own

    for p_len in (-1, 1 << 20):
        good, own = run(p_len=p_len)
        assert good[:2 * n].all() and own[2 * n:].all()
    good, _ = run(page=-3)
    assert good[:2 * n].all()
    good, own = run(p_start=[0, 2 * n, 2 * n - 1])
    assert good[:2 * n - 1].all() and own[2 * n:].all()
    good, own = run(p_start=[0, 2 * n, 4 * n + 1])
    assert good[:2 * n].all() and own[2 * n:].all()
    good, own = run(p_start=[-1, 2 * n, 4 * n])
    assert own[:2 * n].all() and good[2 * n:].all()


def test_broken_sequences_are_left_alone():
    s = Shared([(2, 30)] * 3, [(100, 3)], seed=13)
    s.w.kv_len[1] = 1
    cache, batch, prefix = s.handles()
    q = s.w.randn(s.w.heads)
    o = torch.full_like(q, 7.0)
    P.paged_attend_shared(cache, batch, prefix, q, o)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
    want, _, tol, _ = s.whole.attend(q)
    assert (o[2:4] == 7).all()
    assert ((o.double() - want).abs() <= tol)[[0, 1, 4, 5]].all()


@pytest.mark.parametrize("n", [2, 30])
def test_captured_and_replayed(n):
    """Replays follow the arrays: other lengths of both parts, other bounds, another page table."""
    kw = dict(heads=8, kv_heads=2, seed=14)
    a = Shared([(2, 40)] * n, [(500, n)], **kw)
    w = a.w
    cache, batch, prefix = a.handles()
    q, o = w.randn(w.heads), torch.empty(w.rows, w.heads, w.dim, dtype=w.dtype, device="cuda")
    ws = torch.empty(P.paged_attend_shared_workspace(cache, batch, prefix, w.rows, w.heads), dtype=torch.uint8, device="cuda")
    call = lambda: P.paged_attend_shared(cache, batch, prefix, q, o, workspace=ws)     # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for length, half in ((500, n), (17, n), (300, n // 2)):
        b = Shared([(2, 40)] * n, [(500, n)], **kw)
        w.kv_len[n] = length
        a.p_start[1] = 2 * half
        for j in range(n):
            k = length if j < half else 0
            b.whole.lens[j] = (2, k + 40)
            b.whole.K[j], b.whole.V[j] = (torch.cat([x[n][:k], x[j]]) for x in (b.w.K, b.w.V))
        q.copy_(w.randn(w.heads))
        o.fill_(7.0)
        ws.fill_(255)                                # nothing is kept between calls
        graph.replay()
        assert P.paged_device_error() == 0
        want, _, tol, _ = b.whole.attend(q)
        assert ((o.double() - want).abs() <= tol).all()


def test_two_streams_at_once():
    worlds = [Shared([(1, 50)] * 20, [(900, 20)], seed=15), Shared([(9, 50)] * 7, [(400, 7)], seed=16)]
    jobs = []
    for s in worlds:
        q = s.w.randn(s.w.heads)
        jobs.append((s, q, torch.empty_like(q), s.handles(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _, q, o, handles, stream in jobs:
        P.paged_attend_shared(*handles, q, o, stream=stream)
    assert P.paged_device_error() == 0
    for s, q, o, _, _ in jobs:
        want, _, tol, _ = s.whole.attend(q)
        assert ((o.double() - want).abs() <= tol).all()


def test_the_same_call_gives_the_same_bits():
    s = Shared([(1, 50)] * 33, [(2000, 33)], seed=17)
    q = s.w.randn(s.w.heads)
    handles, got = s.handles(), []
    for _ in range(3):
        o = torch.empty_like(q)
        P.paged_attend_shared(*handles, q, o)
        got.append(o.view(torch.int16))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_a_call_keeps_its_own_workspace_until_it_is_launched(monkeypatch):
    """Another thread's allocations in front of the launch must not find it free."""
    s = Shared([(1, 50)] * 33, [(2000, 33)], seed=18)
    q = s.w.randn(s.w.heads)
    o = torch.empty_like(q)
    cache, batch, prefix = s.handles()
    lib, seen = P._load(), []

    class Watched:
        def __getattr__(self, name):
            f = getattr(lib, name)
            if name.endswith("workspace"):
                return f
            return lambda *a: (seen.append(torch.cuda.memory_allocated()), f(*a))[1]

    monkeypatch.setattr(P, "_load", Watched)
    for call, size in ((lambda: P.paged_attend(cache, batch, q, o), P.paged_attend_workspace(cache, batch, s.w.heads)),
                       (lambda: P.paged_attend_shared(cache, batch, prefix, q, o),
                        P.paged_attend_shared_workspace(cache, batch, prefix, s.w.rows, s.w.heads))):
        before = torch.cuda.memory_allocated()
        del seen[:]
        call()
        assert len(seen) == 1 and seen[0] >= before + size
    monkeypatch.undo()
    assert P.paged_device_error() == 0
