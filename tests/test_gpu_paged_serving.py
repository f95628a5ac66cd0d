"""The paged operators together, as a serving loop runs them: prompt chunks, drafted blocks with
rollback, graphs, streams."""

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from speculative_decoding_draft_kv_gb300 import ring as R
from tests.paged_oracle import World, norm_rope

pytestmark = pytest.mark.gpu


class Loop:
    """Sequences that grow through append + attend, beside their own true history."""

    def __init__(self, n_seq, fmt, dtype, heads=8, kv_heads=2, dim=128, page=16, cap=640, seed=0):
        per = cap // page
        self.w = World([(1, cap)] * n_seq, page=page, heads=heads, kv_heads=kv_heads, dim=dim, fmt=fmt, dtype=dtype, seed=seed,
                       fill=False)
        self.len = [0] * n_seq
        self.hist = [[torch.empty(0, kv_heads, dim, dtype=torch.float64, device="cuda")] * 2 for _ in range(n_seq)]
        self.rope = P.PagedRope(dim, 1e6)
        self.wq, self.wk = (1 + 0.1 * torch.randn(dim, generator=self.w.g, device="cuda") for _ in range(2))
        self.cap = per * page

    def step(self, new, stream=None):
        w = self.w
        lens = [(n, l + n) for n, l in zip(new, self.len)]
        w.lens = lens
        w.q_start.copy_(torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32))
        w.kv_len.copy_(torch.tensor([kv for _, kv in lens], dtype=torch.int32))
        w.total = w.rows = sum(new)
        cache, batch = w.handles(P)
        qkv = torch.randn(w.rows, w.heads + 2 * w.kv_heads, w.dim, generator=w.g, device="cuda").to(w.dtype)
        q, k, v = qkv[:, :w.heads], qkv[:, w.heads:w.heads + w.kv_heads], qkv[:, w.heads + w.kv_heads:]
        qr, o = torch.empty(w.rows, w.heads, w.dim, dtype=w.dtype, device="cuda"), torch.empty(w.rows, w.heads, w.dim, dtype=w.dtype, device="cuda")
        P.paged_append(cache, batch, k, v, rope=self.rope, k_norm=self.wk, q=q, q_norm=self.wq, q_out=qr)
        P.paged_attend(cache, batch, qr, o)
        back = [torch.empty(w.rows, w.kv_heads, w.dim, dtype=w.dtype, device="cuda") for _ in range(2)]
        P.paged_gather(cache, batch, *back)
        assert P.paged_device_error() == 0
        pos = torch.cat([torch.arange(l, l + n) for n, l in zip(new, self.len)]).int().cuda()
        want_k = norm_rope(k, pos, self.wk, 1e-6, self.rope)
        # what a row of the cache may be off by: the type's half step, int8 half a code of the largest
        # value, e4m3 2^-4 of the value
        unit = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}.get(w.fmt)
        for got, want in ((back[0], want_k), (back[1], v.double())):
            top = want.abs().amax(-1, keepdim=True)
            tol = unit * want.abs() if unit else (top / 254 if w.fmt == "int8" else want.abs() * 2.0 ** -4 + top * 2.0 ** -18)
            half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[w.dtype]
            assert ((got.double() - want).abs() <= tol + (half * 1.07 + 2.0 ** -18) * top + 1e-9).all()
        # attention over what the cache really holds: its rows as gathered
        at = 0
        w.K, w.V = [], []
        for s, n in enumerate(new):
            kv = self.exact_rows(s, self.len[s] + n)
            w.K.append(kv[0])
            w.V.append(kv[1])
            at += n
        want, _, tol, _ = w.attend(qr, wide=max(new) * w.heads > 32 * w.kv_heads)
        assert ((o.double() - want).abs() <= tol).all(), float(((o.double() - want).abs() / tol).max())
        self.len = [l + n for n, l in zip(new, self.len)]
        return o

    def exact_rows(self, s, kv):
        w = self.w
        p = torch.arange(kv, device="cuda")
        page, slot = w.pages[s][p // w.page].long(), p % w.page
        if w.ks is None:
            return w.k[page, :, slot].double(), w.v[page, :, slot].double()
        return [pool.view(torch.uint8)[page, :, slot].view(pool.dtype).double() * sc[page, :, slot].double()[..., None]
                for pool, sc in ((w.k, w.ks), (w.v, w.vs))]

    def roll_back(self, keep):
        self.len = [l - k for l, k in zip(self.len, keep)]


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("e4m3", "bf16")])
def test_prompt_then_drafted_blocks_with_rollback(fmt, dtype):
    """Prompt chunks of uneven length, then blocks of 9 of which a part is taken back each time."""
    loop = Loop(3, fmt, dtype)
    loop.step([100, 1, 37])
    loop.step([130, 64, 1])
    for t in range(4):
        loop.step([9, 9, 9])
        loop.roll_back([(t + 3 * i) % 9 for i in range(3)])
    loop.step([1, 1, 1])
    loop.step([200, 0, 1])


def test_same_call_same_bits():
    for lens in ([(9, 5000), (1, 300)], [(300, 2000), (1, 3000)]):
        w = World(lens, seed=21)
        cache, batch = w.handles(P)
        q = w.randn(w.heads)
        outs = []
        for _ in range(3):
            o = torch.empty_like(q)
            P.paged_attend(cache, batch, q, o)
            outs.append(o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("n", [4, 70])
def test_captured_step_follows_its_arrays(n):
    """A captured append + attend, replayed after lengths, pages and rows changed."""
    w = World([(n, 310), (n, 250)], seed=22)               # every length below stays within written rows
    rope = P.PagedRope(128, 1e6)
    q, k, v = w.randn(w.heads), w.randn(w.kv_heads), w.randn(w.kv_heads)
    qo, o = torch.empty_like(q), torch.empty_like(q)
    cache, batch = w.handles(P)
    ws = torch.empty(P.paged_attend_workspace(cache, batch, w.heads), dtype=torch.uint8, device="cuda")

    def step():
        P.paged_append(cache, batch, k, v, rope=rope, q=q, q_out=qo)
        P.paged_attend(cache, batch, qo, o, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    own = torch.cuda.CUDAGraph()
    o_own = torch.empty_like(q)
    with torch.cuda.graph(own):                            # a workspace of the graph's own pool
        P.paged_attend(cache, batch, qo, o_own)
    for lens in ([(n, 301), (n, 88)], [(n, n), (n, 200)], [(n - 1, 250), (2, 2)]):
        w.lens = lens
        w.total = sum(a for a, _ in lens)
        w.q_start.copy_(torch.tensor([0, lens[0][0], w.total], dtype=torch.int32))
        w.kv_len.copy_(torch.tensor([b for _, b in lens], dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=w.g, device="cuda"))
        graph.replay()
        own.replay()
        got, got_own = o[:w.total].clone(), o_own[:w.total].clone()
        o2, qo2 = torch.empty_like(o), torch.empty_like(qo)
        P.paged_append(cache, batch, k, v, rope=rope, q=q, q_out=qo2)
        P.paged_attend(cache, batch, qo2, o2)
        assert torch.equal(got, o2[:w.total]) and torch.equal(got_own, got)
    assert P.paged_device_error() == 0


def test_calls_on_other_streams():
    """Two streams at once, each with its own outputs and workspace."""
    worlds = [World([(9, 3000), (1, 2000)], seed=23), World([(200, 1500)], seed=24)]
    qs = [w.randn(w.heads) for w in worlds]
    hs = [w.handles(P) for w in worlds]
    want = []
    for w, q, h in zip(worlds, qs, hs):
        o = torch.empty_like(q)
        P.paged_attend(*h, q, o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in worlds]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for i in range(20):
        for st, q, h, o in zip(streams, qs, hs, outs):
            if i % 2:
                P.paged_attend(*h, q, o[i], stream=st)
            else:
                with torch.cuda.stream(st):
                    P.paged_attend(*h, q, o[i])
    torch.cuda.synchronize()
    for o, x in zip(outs, want):
        assert all(torch.equal(y, x) for y in o)


def test_refusals():
    w = World([(2, 40)], seed=25)
    cache, batch = w.handles(P)
    q = w.randn(w.heads)
    o = torch.empty_like(q)
    bad = [
        lambda: P.paged_attend(cache, batch, q.float(), o), lambda: P.paged_attend(cache, batch, q.bfloat16(), o.bfloat16()),
        lambda: P.paged_attend(cache, batch, q, o[:1]), lambda: P.paged_attend(cache, batch, q.cpu(), o),
        lambda: P.paged_attend(cache, batch, q[..., :64], o[..., :64]), lambda: P.paged_attend(cache, batch, q, o, mask="tree"),
        lambda: P.paged_attend(cache, batch, q, o, mask="none"), lambda: P.paged_attend(cache, batch, q, o, window=-1),
        lambda: P.paged_attend(cache, batch, q, o, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: P.paged_attend(cache, batch, q, o, lse=torch.empty(1, device="cuda")),
        lambda: P.paged_append(cache, batch, q, q), lambda: P.paged_gather(cache, batch, q, q),
        lambda: P.PagedCache(w.k, w.v.bfloat16()), lambda: P.PagedCache(w.k.float(), w.v.float()),
        lambda: P.PagedCache(w.k, w.v, torch.empty(1, device="cuda")), lambda: P.PagedCache(w.k.cpu(), w.v.cpu()),
        lambda: P.PagedBatch(w.q_start.long(), w.kv_len, w.pages, 2), lambda: P.PagedBatch(w.q_start, w.kv_len, w.pages[0], 2),
        lambda: P.paged_norm_rope(None, None), lambda: P.paged_norm_rope(None, None, q=q),
        lambda: P.paged_norm_rope(None, P.PagedRope(128), q=q, q_out=o),
        lambda: P.paged_norm_rope(torch.zeros(1, dtype=torch.int32, device="cuda"), P.PagedRope(128), q=q, q_out=o),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, R.RingError, KeyError)):
            f()
    assert P.paged_device_error() == 0
