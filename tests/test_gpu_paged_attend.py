"""paged_attend against its float64 form: types, page sizes and orders, head groups, lengths on
both sides of a tile, masks that leave rows empty, and what must not matter (NaN in unseen
places, rows behind the batch)."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import World

pytestmark = pytest.mark.gpu

FORMATS = [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("int8", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")]


def trees(w, seed=1, empty=()):
    """A random ancestor set for every row (itself included); rows of `empty` see nothing new."""
    g = torch.Generator().manual_seed(seed)
    words = []
    for n, _ in w.lens:
        for j in range(n):
            bits = int(torch.randint(0, 1 << 62, (1,), generator=g)) | int(torch.randint(0, 4, (1,), generator=g)) << 62
            words.append((bits & ((1 << j) - 1)) | (1 << j))
    words += [0] * (w.rows - w.total)
    for r in empty:
        words[r] = 0
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in words], dtype=torch.int64, device="cuda")


def check(w, mask="causal", window=0, tree=None, scale=None, q=None, max_q=None, stride=None, lse=True):
    q = w.randn(w.heads) if q is None else q
    cache, batch = w.handles(P, max_q)
    o = torch.full((w.rows, w.heads, w.dim), 7.0, dtype=w.dtype, device="cuda")
    if stride:                                   # heads inside a wider row
        wide = torch.full((w.rows, w.heads + 3, w.dim + 8), 7.0, dtype=w.dtype, device="cuda")
        o = wide[:, 1:1 + w.heads, :w.dim]
    ls = torch.full((w.rows, w.heads), 7.0, device="cuda") if lse else None
    P.paged_attend(cache, batch, q, o, mask=mask, window=window, scale=scale or 0.0, tree=tree, lse=ls)
    wide = max(n for n, _ in w.lens) * (w.heads // w.kv_heads) > 32 if max_q is None else max_q * w.heads > 32 * w.kv_heads
    want, wl, tol, ltol = w.attend(q, mask, window, tree, scale, wide)
    assert P.paged_device_error() == 0
    got = o[:w.total].double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got - want).abs() / tol).max()))
    assert (o[w.total:] == 7.0).all(), "rows behind the batch"
    if lse:
        gl = ls[:w.total].double()
        none = torch.isinf(wl)
        assert torch.equal(gl[none], wl[none])
        assert ((gl - wl)[~none].abs() <= ltol[~none]).all(), float(((gl - wl).abs() / ltol)[~none].max())
        assert (ls[w.total:] == 7.0).all()
    return o


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 63), (1, 64), (1, 65), (1, 129)], [(4, 4), (3, 200), (1, 1000)], [(8, 777), (0, 50), (5, 5)],
    [(40, 300), (1, 17), (129, 400)],
])
def test_types_and_lengths(fmt, dtype, dim, lens):
    check(World(lens, fmt=fmt, dtype=dtype, dim=dim, spare_rows=3, seed=len(lens) + dim))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fmt,order", [("f16", "hnd"), ("f16", "nhd"), ("int8", "nhd"), ("e4m3", "hnd")])
def test_pages(page, fmt, order):
    check(World([(2, 2 * page + 1), (3, page - 1), (1, 5 * page), (17, 300)], page=page, fmt=fmt, order=order, seed=page))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (7, 1), (10, 2), (32, 8), (64, 1), (33, 3)])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_head_groups(heads, kv_heads, n):
    check(World([(n, 333), (n, n)], heads=heads, kv_heads=kv_heads, seed=heads + n))


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("window", [1, 5, 64, 100])
@pytest.mark.parametrize("mask", ["causal", "full", "tree"])
def test_windows(fmt, dtype, window, mask):
    w = World([(6, 500), (1, 30), (33, 190), (2, 2)], fmt=fmt, dtype=dtype, seed=window)
    check(w, mask, window, trees(w) if mask == "tree" else None)


@pytest.mark.parametrize("window", [1, 70])
def test_pages_in_front_of_the_window_are_not_looked_at(window):
    w = World([(1, 900), (4, 640)], seed=3)
    for s, (n, kv) in enumerate(w.lens):
        first = (kv - n - window + 1) // w.page
        w.pages[s, :max(0, first)] = -1
    check(w, "causal", window)


@pytest.mark.parametrize("fmt,dtype", FORMATS)
def test_trees(fmt, dtype):
    w = World([(31, 400), (64, 64), (1, 1), (64, 200), (9, 137)], fmt=fmt, dtype=dtype, spare_rows=2, seed=5)
    check(w, "tree", 0, trees(w))


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("e4m3", "bf16")])
def test_rows_that_see_nothing(fmt, dtype):
    """No context and no tree bits: zeros and -inf, although the tile holds NaN elsewhere."""
    w = World([(5, 5), (40, 40)], fmt=fmt, dtype=dtype, seed=6)
    o = check(w, "tree", 0, trees(w, empty=(0, 3, 7, 44)))
    assert (o[[0, 3, 7, 44]] == 0).all()


def test_nodes_that_no_token_sees_may_hold_anything():
    for fmt in ("f16", "int8", "e4m3"):
        w = World([(12, 100)], fmt=fmt, seed=7)
        t = trees(w)
        t &= ~(1 << 4)                           # nobody sees node 4, itself included
        p = 100 - 12 + 4
        page, slot = int(w.pages[0, p // w.page]), p % w.page
        if fmt == "f16":
            w.k[page, :, slot] = math.inf
            w.v[page, :, slot] = math.nan
        else:
            w.ks[page, :, slot] = math.nan
            w.vs[page, :, slot] = math.inf
            w.v.view(torch.uint8)[page, :, slot] = 0x7f
        check(w, "tree", 0, t)


@pytest.mark.parametrize("n", [1, 40])
def test_full_mask(n):
    check(World([(n, 150), (n, n), (7, 65)], seed=n), "full")


@pytest.mark.parametrize("n", [4, 60])
def test_strided_queries_and_outputs(n):
    w = World([(n, 200), (2, 70)], seed=11)
    qkv = torch.randn(w.rows, w.heads + 2 * w.kv_heads, w.dim, generator=w.g, device="cuda").half()
    check(w, q=qkv[:, :w.heads], stride=True)


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("n", [2, 50])
def test_wide_scores(fmt, dtype, n):
    """Scores over a hundred units apart: the reference maximum has to follow."""
    w = World([(n, 700), (1, 80)], fmt=fmt, dtype=dtype, seed=12, spread=3.0)
    q = w.randn(w.heads, spread=6.0)
    check(w, q=q)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scales_of_all_sizes(fmt):
    """Scales from 1e-12 to 1e6 side by side; bf16 queries far outside F16's range."""
    w = World([(3, 300), (50, 90)], fmt=fmt, dtype="bf16", seed=13)
    for s, (_, kv) in enumerate(w.lens):
        f = torch.exp(torch.empty(kv, w.kv_heads, device="cuda", dtype=torch.float64).uniform_(-27, 14, generator=w.g)).float()
        p = torch.arange(kv, device="cuda")
        page, slot = w.pages[s][p // w.page].long(), p % w.page
        old = w.vs[page, :, slot]
        w.vs[page, :, slot] = old * f
        w.V[s] = w.V[s] * ((old * f).double() / old.double())[..., None]
    q = w.randn(w.heads, spread=3e6)
    check(w, q=q, scale=1e-7)


def test_a_scale_of_its_own_and_a_loose_bound():
    check(World([(3, 100), (1, 40)], seed=14), scale=0.3, max_q=64)


def test_many_sequences():
    lens = [(1 + i % 3, 1 + (i * 37) % 200 + 3) for i in range(300)]
    check(World(lens, heads=4, kv_heads=1, dim=64, seed=15))


def test_one_long_sequence_among_short_ones():
    check(World([(1, 5)] * 20 + [(2, 9000)] + [(1, 30)] * 7, seed=16))


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("n,long", [(1, 4), (9, 4), (40, 4), (70, 3)])
def test_many_tiles_and_items_a_cta(fmt, dtype, n, long):
    """Enough work that every CTA's stages come round several times, with whole items of one tile
    between long ones."""
    lens = [(1 + (i * 7) % n, 1 + (i * 7) % n + (i * 611) % (1200 * (1 if i % long else 4))) for i in range(48)]
    check(World(lens, heads=32, kv_heads=8, page=32, fmt=fmt, dtype=dtype, seed=n))


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("e4m3", "bf16")])
def test_every_item_of_one_tile(fmt, dtype):
    lens = [(1 + i % 35, 1 + i % 35 + (i * 13) % 80) for i in range(150)]
    check(World(lens, heads=32, kv_heads=8, page=16, fmt=fmt, dtype=dtype, seed=3))


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("n", [3, 40])
def test_rows_of_zeros_and_tiny_scales(fmt, dtype, n):
    """Queries of zeros weigh what they see alike; a scale next to nothing does the same."""
    w = World([(n, 200), (n, n)], fmt=fmt, dtype=dtype, seed=17)
    q = w.randn(w.heads)
    q[1] = 0
    q[n, 2] = 0
    check(w, q=q)
    check(w, q=q, scale=1e-30)
