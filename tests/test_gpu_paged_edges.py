"""The corners of the paged operators: pools beyond 32-bit offsets, bounds that the arrays break,
windows without end, empty batches, infinities next to a rotation, tensors of no stride, shared
pages, streams given by number, and a capture before any other call."""

import os
import subprocess
import sys

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import build as B
from speculative_decoding_draft_kv_gb300 import paged as P
from speculative_decoding_draft_kv_gb300 import ring as R
from tests.paged_oracle import World
from tests.test_gpu_paged_attend import check, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,n", [("f16", 3), ("f16", 40), ("int8", 3), ("e4m3", 40)])
def test_pages_beyond_32_bit_offsets(fmt, n):
    """The same rows in a small pool and at the end of one whose byte offsets pass 2^32 (its element
    offsets 2^31 in 16-bit formats, 2^32 in codes): the same bits everywhere."""
    w = World([(n, 700), (1, 300)], page=256, fmt=fmt, seed=31)
    q, k, v = w.randn(w.heads), w.randn(w.kv_heads), w.randn(w.kv_heads)
    rope = P.PagedRope(128, 1e6)
    shift = (2 ** 31 if fmt == "f16" else 2 ** 32) // (w.kv_heads * w.page * w.dim)

    def run():
        cache, batch = w.handles(P)
        P.paged_append(cache, batch, k, v, rope=rope)
        outs = [torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)]
        P.paged_gather(cache, batch, outs[0], outs[1])
        P.paged_attend(cache, batch, q, outs[2])
        assert P.paged_device_error() == 0
        return outs

    small = (w.k, w.v, w.ks, w.vs)
    want = run()

    def far(x):
        if x is None:
            return None
        y = torch.empty((shift + w.n_pages,) + x.shape[1:], dtype=x.dtype, device="cuda")
        as_bytes = (lambda t: t) if x.element_size() > 1 else (lambda t: t.view(torch.uint8))
        as_bytes(y)[shift:] = as_bytes(x)
        return y

    w.k, w.v, w.ks, w.vs = (far(x) for x in small)
    w.pages += shift * (w.pages >= 0)
    got = run()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    for x, y in zip(small, (w.k, w.v, w.ks, w.vs)):        # and the same rows were written
        if x is not None:
            kind = torch.int32 if x.dtype == torch.float32 else (torch.int16 if x.element_size() == 2 else torch.uint8)
            assert torch.equal(x.view(kind), y[shift:].view(kind))


@pytest.mark.parametrize("heads,bound", [(8, 3), (8, 20), (16, 40)])
def test_a_sequence_above_max_q_is_left_alone(heads, bound):
    w = World([(2, 90), (bound + 1, 200), (bound, 150)], heads=heads, seed=32)
    cache, batch = w.handles(P, max_q=bound)
    q = w.randn(heads)
    o = torch.full_like(q, 7.0)
    lse = torch.full((w.rows, heads), 7.0, device="cuda")
    P.paged_attend(cache, batch, q, o, lse=lse)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
    skipped = slice(2, bound + 3)
    assert (o[skipped] == 7.0).all() and (lse[skipped] == 7.0).all()
    want, wl, tol, ltol = w.attend(q)
    served = torch.ones(w.rows, dtype=torch.bool, device="cuda")
    served[skipped] = False
    assert ((o.double() - want).abs() <= tol)[served].all()
    assert ((lse.double() - wl).abs() <= ltol)[served].all()


@pytest.mark.parametrize("mask", ["causal", "full", "tree"])
@pytest.mark.parametrize("n", [5, 50])
def test_a_window_past_everything_is_none(mask, n):
    w = World([(n, 300), (1, 1), (n, n)], seed=33)
    tree = trees(w) if mask == "tree" else None
    cache, batch = w.handles(P)
    q = w.randn(w.heads)
    outs = []
    for window in (0, 300, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 300, 2 ** 31 - 1):
        o = torch.empty_like(q)
        P.paged_attend(cache, batch, q, o, mask=mask, window=window, tree=tree)
        outs.append(o)
    assert P.paged_device_error() == 0
    for o in outs[1:]:
        assert torch.equal(outs[0], o)
    with pytest.raises(ValueError):
        P.paged_attend(cache, batch, q, o, mask=mask, window=2 ** 32 + 5, tree=tree)
    with pytest.raises(ValueError):
        P.PagedBatch(w.q_start, w.kv_len, w.pages, 2 ** 32 + 5)


@pytest.mark.parametrize("lens", [[], [(0, 0)], [(0, 40), (0, 0), (0, 17)]])
def test_batches_without_rows(lens):
    base = World(lens or [(0, 1)], seed=34)
    n = len(lens)
    cache = P.PagedCache(base.k, base.v)
    batch = P.PagedBatch(base.q_start[:n + 1], base.kv_len[:n], base.pages[:n], 8)
    for rows in (0, 3):                                    # 3: all of them behind the batch
        q = torch.randn(rows, base.heads, base.dim, device="cuda").half()
        k, v = (torch.full((rows, base.kv_heads, base.dim), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        o, qo = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
        pools = base.k.clone()
        P.paged_append(cache, batch, k, v, rope=P.PagedRope(128), q=q, q_out=qo)
        P.paged_gather(cache, batch, k, v)
        P.paged_attend(cache, batch, q, o)
        assert P.paged_device_error() == 0
        assert (o == 7).all() and (qo == 7).all() and (k == 7).all() and (v == 7).all()
        assert torch.equal(pools.view(torch.int16), base.k.view(torch.int16))
    none = torch.empty(0, 4, 128, device="cuda")
    P.paged_norm_rope(torch.empty(0, dtype=torch.int32, device="cuda"), P.PagedRope(128), q=none, q_out=none)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_infinities_stay_in_their_pair(layout, dtype):
    """An infinity in an element that is not turned is one after it, and every other element is as if
    it were not there; one in a pair stays in the pair."""
    r = P.PagedRope(64, 1e4, layout)
    x = torch.randn(9, 3, 128, device="cuda").to(dtype)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 77 + 1
    bad = x.clone()
    bad[:, 0, 64:72] = float("inf")
    bad[:, 1, 127] = -float("inf")
    bad[:, 2, 40] = float("inf")
    y = torch.empty_like(bad)
    P.paged_norm_rope(pos, r, q=bad, q_out=y)
    assert (y[:, 0, 64:72] == float("inf")).all() and (y[:, 1, 127] == -float("inf")).all()
    touched = torch.zeros(3, 128, dtype=torch.bool, device="cuda")
    touched[0, 64:72] = touched[1, 127] = touched[2, 40] = touched[2, 8 if layout == "half" else 41] = True
    assert not torch.isfinite(y[:, 2, 40]).any()
    y = torch.where(touched, torch.zeros_like(y), y)
    assert torch.isfinite(y).all()
    plain = torch.empty_like(x)
    P.paged_norm_rope(pos, r, q=x, q_out=plain)
    assert torch.equal(y, torch.where(touched, torch.zeros_like(plain), plain))


def test_tensors_of_no_stride_and_in_place():
    w = World([(4, 40)], seed=35)
    cache, batch = w.handles(P)
    q, k, v = w.randn(w.heads), w.randn(w.kv_heads), w.randn(w.kv_heads)
    o = torch.empty_like(q)
    rope, pos = P.PagedRope(128), torch.arange(4, dtype=torch.int32, device="cuda")
    wider = torch.empty(4, w.heads + 1, 128, dtype=q.dtype, device="cuda")
    bad = [
        lambda: P.paged_attend(cache, batch, q[:1].expand(4, -1, -1), o),
        lambda: P.paged_attend(cache, batch, q, o[:, :1].expand(-1, w.heads, -1)),
        lambda: P.paged_attend(cache, batch, q, q),
        lambda: P.paged_append(cache, batch, k[:, :1].expand(-1, w.kv_heads, -1), v),
        lambda: P.paged_gather(cache, batch, k[:1].expand(4, -1, -1), v),
        lambda: P.paged_norm_rope(pos, rope, q=q, q_out=o[:1].expand(4, -1, -1)),
        lambda: P.paged_norm_rope(pos, rope, q=wider.view(-1)[:q.numel()].view_as(q), q_out=wider[:, :w.heads]),
        lambda: P.paged_append(cache, batch, k, v, rope=rope, q=wider.view(-1)[:q.numel()].view_as(q), q_out=wider[:, :w.heads]),
    ]
    for f in bad:
        with pytest.raises((ValueError, R.RingError)):
            f()
    want = torch.empty_like(q)
    P.paged_append(cache, batch, k, v, rope=rope, q=q, q_out=want)
    P.paged_append(cache, batch, k, v, rope=rope, q=q, q_out=q)       # in its own place
    assert torch.equal(q, want)


@pytest.mark.parametrize("n", [3, 40])
def test_sequences_that_share_pages(n):
    """A common beginning held once: two block tables that name the same pages."""
    w = World([(n, 300), (n, 300), (1, 128)], page=32, seed=36)
    w.pages[1] = w.pages[0]
    w.pages[2, :4] = w.pages[0, :4]
    w.K[1], w.V[1] = w.K[0], w.V[0]
    w.K[2], w.V[2] = w.K[0][:128], w.V[0][:128]
    check(w)
    check(w, "full")


def test_streams_by_number():
    """A stream may be None, PyTorch's or a handle (0: the default stream), also where the call makes
    its own workspace and another stream is the current one."""
    w = World([(9, 3000), (1, 2000)], seed=37)
    cache, batch = w.handles(P)
    q = w.randn(w.heads)
    want = torch.empty_like(q)
    P.paged_attend(cache, batch, q, want)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for stream in (0, side, side.cuda_stream, None) * 5:
            o = torch.empty_like(q)
            other.synchronize()
            P.paged_attend(cache, batch, q, o, stream=stream)
            outs.append(o)
            # what would fill a workspace that was taken from the wrong stream's memory
            torch.full((P.paged_attend_workspace(cache, batch, w.heads),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_graphs_that_share_a_workspace_one_after_another():
    worlds = [World([(3, 2500)], seed=38), World([(60, 900), (1, 1200)], seed=39)]
    hs, qs = [w.handles(P) for w in worlds], [w.randn(w.heads) for w in worlds]
    size = max(P.paged_attend_workspace(*h, w.heads) for h, w in zip(hs, worlds))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want, outs, graphs = [], [torch.empty_like(q) for q in qs], []
    for h, q in zip(hs, qs):
        want.append(torch.empty_like(q))
        P.paged_attend(*h, q, want[-1])
    torch.cuda.synchronize()
    for h, q, o in zip(hs, qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            P.paged_attend(*h, q, o, workspace=ws)
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_captured_before_any_other_call():
    """A process whose first calls of these operators are captured ones."""
    code = """
import torch
from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import World
w = World([(3, 300), (60, 200)])
cache, batch = w.handles(P)
rope = P.PagedRope(128)
q, k, v = w.randn(8), w.randn(2), w.randn(2)
qo, o, o2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    P.paged_append(cache, batch, k, v, rope=rope, q=q, q_out=qo)
    P.paged_attend(cache, batch, qo, o)
g.replay()
P.paged_attend(cache, batch, qo, o2)
assert P.paged_device_error() == 0 and torch.equal(o, o2) and bool(torch.isfinite(o).all())
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=B.ROOT, env=dict(os.environ, PYTHONPATH=B.ROOT), timeout=300)
