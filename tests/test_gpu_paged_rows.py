"""paged_norm_rope, paged_append and paged_gather against their float64 forms, bit for bit where
nothing rounds twice."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import FORMATS, TOP, UNIT, World, norm_rope

pytestmark = pytest.mark.gpu

ROPES = {
    "none": None,
    "half128": dict(rotary_dim=128, theta=1e6),
    "half64": dict(rotary_dim=64, theta=1e4),
    "half48": dict(rotary_dim=48, theta=1e6, scaling="linear", factor=4.0),
    "inter64": dict(rotary_dim=64, theta=1e6, layout="interleaved", scaling="yarn", factor=8.0, original_len=4096),
    "inter16": dict(rotary_dim=16, theta=1e4, layout="interleaved", scaling="ntk", factor=8.0),
    "inter128": dict(rotary_dim=128, theta=1e4, layout="interleaved"),
}


def rope_of(name, dim):
    if ROPES[name] is None:
        return None
    d = dict(ROPES[name])
    d["rotary_dim"] = min(d["rotary_dim"], dim)
    return P.PagedRope(**d)


def amplitude(y, x, positions, w, eps, rope):
    """What an element's float32 roundings are relative to: of a pair, |x1| + |x2| after the norm."""
    flat = norm_rope(x, positions, w, eps, None).abs()
    if rope is None:
        return flat
    r = rope.args.rotary_dim
    a = flat.clone()
    one, two = (slice(0, r // 2), slice(r // 2, r)) if rope.args.layout == 0 else (slice(0, r, 2), slice(1, r, 2))
    a[..., one] = a[..., two] = (flat[..., one] + flat[..., two]) * rope.magnitude
    return a


#: The norm rounds 12 times in its sum (halved by the root), twice in the root (2 ulp) and twice in
#: the products: 10 half steps of 2^-24.  An angle is off by 2^-25 of a turn (its fraction in 24
#: bits), 1.9e-7, sincospif by under 2^-22, and the rotation rounds twice more.  All below 2^-20.
ROUND = 2.0 ** -20


def near(got, x, positions, w, eps, rope, unit):
    want = norm_rope(x, positions, w, eps, rope)
    tol = unit * want.abs() + ROUND * amplitude(want, x, positions, w, eps, rope) + 2.0 ** -25
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), float(((got.double() - want).abs() / tol).max()))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("rows,heads,kv_heads", [(1, 1, 1), (3, 32, 8), (700, 7, 3)])
def test_norm_rope(dtype, dim, rope, rows, heads, kv_heads):
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    qkv = torch.randn(rows, heads + 2 * kv_heads, dim, generator=g, device="cuda").to(dtype)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv_heads]
    wq, wk = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda") for _ in range(2))
    r = rope_of(rope, dim)
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, device="cuda", dtype=torch.int32)
    pos[-1] = 2 ** 31 - 1 if rows > 1 else 0
    qo, ko = torch.empty(rows, heads, dim, dtype=dtype, device="cuda"), torch.empty(rows, kv_heads, dim, dtype=dtype, device="cuda")
    P.paged_norm_rope(pos, r, 1e-6, q=q, q_norm=wq, q_out=qo, k=k, k_norm=wk, k_out=ko)
    # the last position is 2^31 - 1: inv_freq itself, a float64, is off by up to 2^-53 of it
    # there, 2^31 2^-53 radians, far below ROUND
    near(qo, q, pos, wq, 1e-6, r, UNIT[dtype])
    near(ko, k, pos, wk, 1e-6, r, UNIT[dtype])


def test_norm_rope_one_of_the_two_without_norm_and_in_place():
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(33, 5, 128, generator=g, device="cuda").half()
    pos = torch.arange(33, device="cuda", dtype=torch.int32) * 1000
    r = rope_of("half128", 128)
    was = q.clone()
    P.paged_norm_rope(pos, r, q=q, q_out=q)
    near(q, was, pos, None, 1e-6, r, UNIT[q.dtype])
    k = torch.empty_like(was)
    P.paged_norm_rope(None, None, k=was, k_out=k)          # neither norm nor rotation: a copy
    assert torch.equal(k, was)


def test_rotation_at_zero_is_the_identity_and_zeros_stay():
    x = torch.randn(4, 2, 64, device="cuda")
    y = torch.empty_like(x)
    r = P.PagedRope(64, 1e4)
    P.paged_norm_rope(torch.zeros(4, dtype=torch.int32, device="cuda"), r, q=x, q_out=y)
    assert torch.equal(x, y)
    z = torch.zeros_like(x)
    P.paged_norm_rope(torch.arange(4, dtype=torch.int32, device="cuda"), r, eps=1e-6, q=z, q_out=y,
                      q_norm=torch.ones(64, device="cuda"))
    assert (y == 0).all()


def places(w, s):
    n, kv = w.lens[s]
    p = torch.arange(kv - n, kv, device="cuda")
    return w.pages[s][p // w.page].long(), p % w.page


def snapshot(w):
    return [t.clone() for t in (w.k.view(torch.uint8), w.v.view(torch.uint8)) + ((w.ks.view(torch.int32), w.vs.view(torch.int32)) if w.ks is not None else ())]


def only_changed(w, before):
    """Nothing but the batch's own places changed."""
    touched = torch.zeros(w.n_pages, w.page, dtype=torch.bool, device="cuda")
    for s in range(len(w.lens)):
        page, slot = places(w, s)
        touched[page, slot] = True
    for old, new in zip(before, snapshot(w)):
        same = (old == new).reshape(w.n_pages, w.kv_heads, w.page, -1).all(-1).all(1)
        assert (same | touched).all()


LENS = [[(1, 1)], [(9, 9), (1, 100), (0, 40), (16, 31)], [(130, 300), (2, 17)], [(1, 1 + 7 * i) for i in range(70)]]


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("int8", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("dim,page,order", [(128, 16, "hnd"), (64, 64, "nhd")])
@pytest.mark.parametrize("lens", LENS)
def test_append_writes_the_rows_bit_for_bit(fmt, dtype, dim, page, order, lens):
    """Without norm and rotation: the same float32 operations in PyTorch give the same bits."""
    w = World(lens, page=page, dim=dim, fmt=fmt, dtype=dtype, order=order, kv_heads=3, heads=3, spare_rows=4, fill=False)
    k, v = w.randn(3), w.randn(3, spread=5.0)
    v[0, 0] = 0                                            # a row of zeros
    cache, batch = w.handles(P)
    before = snapshot(w)
    P.paged_append(cache, batch, k, v)
    assert P.paged_device_error() == 0
    only_changed(w, before)
    for s, (n, kv) in enumerate(lens):
        page_id, slot = places(w, s)
        r = slice(int(w.q_start[s]), int(w.q_start[s]) + n)
        for pool, scale, x in ((w.k, w.ks, k[r]), (w.v, w.vs, v[r])):
            got = pool.view(torch.uint8)[page_id, :, slot].view(pool.dtype) if scale is not None else pool[page_id, :, slot]
            if scale is None:
                assert torch.equal(got, x)
                continue
            top = x.float().abs().amax(-1, keepdim=True)
            # as a tensor: PyTorch divides by (and into) a plain number through a reciprocal
            full = torch.full_like(top, TOP[w.store])
            y = x.float() * torch.where(top > 0, full / top, 0.0)
            codes = y.round().to(torch.int8) if w.store == torch.int8 else y.to(w.store)
            assert torch.equal(got.view(torch.uint8), codes.view(torch.uint8))
            assert torch.equal(scale[page_id, :, slot], (top / full)[..., 0])


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("rope", ["half128", "inter64", "half48"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("depths", [False, True])
def test_append_norms_and_turns(fmt, dtype, rope, dim, depths):
    lens = [(5, 5), (3, 900), (64, 64), (1, 2)]
    w = World(lens, dim=dim, fmt=fmt, dtype=dtype, spare_rows=2, fill=False)
    r = rope_of(rope, dim)
    q, k, v = w.randn(w.heads), w.randn(w.kv_heads), w.randn(w.kv_heads)
    wq, wk = (1 + 0.2 * torch.randn(dim, generator=w.g, device="cuda") for _ in range(2))
    qo = torch.full_like(q, 7.0)
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in lens] + [torch.zeros(2, dtype=torch.long)]).int().cuda()
    if depths:
        pos = torch.randint(0, 5000, pos.shape, generator=w.g, device="cuda", dtype=torch.int32)
    cache, batch = w.handles(P)
    before = snapshot(w)
    P.paged_append(cache, batch, k, v, rope=r, k_norm=wk, q=q, q_norm=wq, q_out=qo, positions=pos if depths else None)
    assert P.paged_device_error() == 0
    only_changed(w, before)
    t = w.total
    assert (qo[t:] == 7.0).all()
    near(qo[:t], q[:t], pos[:t], wq, 1e-6, r, UNIT[w.dtype])
    want = norm_rope(k[:t], pos[:t], wk, 1e-6, r)
    amp = ROUND * amplitude(want, k[:t], pos[:t], wk, 1e-6, r)
    got_k = torch.empty(w.rows, w.kv_heads, dim, dtype=torch.float64, device="cuda")
    for s, (n, _) in enumerate(lens):
        page_id, slot = places(w, s)
        rr = slice(int(w.q_start[s]), int(w.q_start[s]) + n)
        if w.ks is None:
            got_k[rr] = w.k[page_id, :, slot].double()
            assert torch.equal(w.v[page_id, :, slot], v[rr])
        else:
            got_k[rr] = w.k.view(torch.uint8)[page_id, :, slot].view(w.store).double() * w.ks[page_id, :, slot].double()[..., None]
    off = (got_k[:t] - want).abs()
    if w.ks is None:
        assert (off <= UNIT[w.dtype] * want.abs() + amp + 2.0 ** -25).all()
    else:
        top = want.abs().amax(-1, keepdim=True)
        full = TOP[w.store]
        # half a code step (int8: of the scale; e4m3: 2^-4 of the value, 2^-10 of the scale where
        # it is subnormal), the scale's own rounding, and the value's
        step = 0.5 * top / full if w.store == torch.int8 else torch.maximum(want.abs() * 2.0 ** -4, 2.0 ** -10 * top / full)
        assert (off <= step * (1 + 2.0 ** -16) + 2.0 ** -21 * want.abs() + 2 * amp + amp.amax(-1, keepdim=True)).all(), float((off / step).max())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_with_infinities_read_back_as_nan_and_tiny_ones_as_zeros(fmt):
    w = World([(4, 4)], fmt=fmt, dtype="bf16", fill=False)
    k, v = w.randn(w.kv_heads), w.randn(w.kv_heads)
    k[1, 0, 5] = math.inf
    v[2, 1, 127] = math.nan
    v[3, 0] = 1e-31
    cache, batch = w.handles(P)
    P.paged_append(cache, batch, k, v)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    P.paged_gather(cache, batch, ko, vo)
    assert ko[1, 0].isnan().all() and vo[2, 1].isnan().all() and (vo[3, 0] == 0).all()
    assert ko.isnan().sum() == w.dim and vo.isnan().sum() == w.dim


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("int8", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("dim,page,order", [(128, 16, "nhd"), (64, 256, "hnd"), (128, 32, "hnd")])
@pytest.mark.parametrize("lens", [[(1, 1)], [(33, 33), (0, 5), (700, 700)], [(4, 90), (1, 300)]])
def test_gather(fmt, dtype, dim, page, order, lens):
    w = World(lens, page=page, dim=dim, fmt=fmt, dtype=dtype, order=order, kv_heads=3, heads=3, spare_rows=2)
    cache, batch = w.handles(P)
    wide = torch.full((w.rows, 9, dim + 8), 7.0, dtype=w.dtype, device="cuda")
    k, v = wide[:, 1:4, :dim], wide[:, 5:8, :dim]
    P.paged_gather(cache, batch, k, v)
    assert P.paged_device_error() == 0
    for s, (n, kv) in enumerate(lens):
        r = slice(int(w.q_start[s]), int(w.q_start[s]) + n)
        for got, true in ((k, w.K), (v, w.V)):
            # codes times scale in float32, one rounding more to the type
            want = true[s][kv - n:].float().to(w.dtype)
            off = (got[r].double() - true[s][kv - n:]).abs()
            assert (off <= (UNIT[w.dtype] + 2.0 ** -24) * true[s][kv - n:].abs() + 2.0 ** -25).all()
            if w.ks is None:
                assert torch.equal(got[r], want)
    assert (wide[w.total:] == 7.0).all() and (wide[:, :, dim:] == 7.0).all()
    assert (wide[:, [0, 4, 8]] == 7.0).all()


def test_places_out_of_range_are_not_followed():
    """Page numbers outside the pool, lengths beyond the block table or below the new rows: such
    rows are skipped and read as zeros, the others are served, and the error word says so."""
    lens = [(3, 40), (2, 20), (4, 50), (2, 2)]
    w = World(lens, fill=False)
    k, v = w.randn(w.kv_heads), w.randn(w.kv_heads)
    w.pages[0, 39 // w.page] = w.n_pages                   # positions 32 .. 39: all three rows
    w.pages[1, 19 // w.page] = -1                          # positions 16 .. 19: both rows
    w.kv_len[2] = w.max_pages * w.page + 1                 # no such place
    cache, batch = w.handles(P)
    before = snapshot(w)
    P.paged_append(cache, batch, k, v)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
    assert P.paged_device_error() == 0
    page, slot = places(w, 3)
    changed = torch.zeros(w.n_pages, w.page, dtype=torch.bool, device="cuda")
    changed[page, slot] = True
    for old, new in zip(before, snapshot(w)):
        same = (old == new).reshape(w.n_pages, w.kv_heads, w.page, -1).all(-1).all(1)
        assert torch.equal(same, ~changed)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    P.paged_gather(cache, batch, ko, vo)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
    assert (ko[:9] == 0).all() and (vo[:9] == 0).all()
    assert torch.equal(ko[9:], k[9:]) and torch.equal(vo[9:], v[9:])
    q = w.randn(w.heads)
    o = torch.full_like(q, 7.0)
    w.kv_len[2] = 1                                        # fewer cached than new
    P.paged_attend(cache, batch, q, o)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
    solo = World([(2, 2)], fill=False, seed=9)
    c2, b2 = solo.handles(P)
    P.paged_append(c2, b2, k[9:11], v[9:11])
    o2 = torch.empty_like(q[9:11])
    P.paged_attend(c2, b2, q[9:11], o2)
    assert torch.equal(o[9:11], o2)
