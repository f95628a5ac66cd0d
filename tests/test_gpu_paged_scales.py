"""paged_attend over quantised pages whose rows' scales are far apart: what a query row gets is as exact
as the rows that it sees and weighs, whatever scales it does not see, or sees without weighing them."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import UNIT, World

pytestmark = pytest.mark.gpu

#: A probability times its V scale is an F16 value in a unit of the row's own, at most this many times the
#: largest such product of the row.
UNIT_ABOVE_WEIGHT = 2.0 ** 11


def rescale(w, s, which, factor):
    """The scales of sequence s's K or V rows times factor [kv, kv_heads]."""
    pool, true = (w.ks, w.K) if which == "k" else (w.vs, w.V)
    p = torch.arange(w.lens[s][1], device="cuda")
    page, slot = w.pages[s][p // w.page].long(), p % w.page
    old = pool[page, :, slot]
    new = (old * factor).float()
    pool[page, :, slot] = new
    true[s] = true[s] * (new.double() / old.double())[..., None]


def put_keys(w, s, positions, direction, lengths):
    """K rows of some positions along direction [kv_heads, dim], each of its (signed) length."""
    p, size = torch.as_tensor(positions, device="cuda"), torch.as_tensor(lengths, dtype=torch.float64, device="cuda")
    x = direction / direction.abs().amax(-1, keepdim=True) * 100
    x = x[None] * torch.where(size < 0, -1.0, 1.0)[:, None, None]
    codes = (x.round() if w.store == torch.int8 else x.float()).to(w.store)
    value = codes.double()
    scale = (size.abs()[:, None] / value.square().sum(-1).sqrt()).float()
    page, slot = w.pages[s][p // w.page].long(), p % w.page
    w.k.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
    w.ks[page, :, slot] = scale
    w.K[s][p] = value * scale.double()[..., None]


def queries(w, spread=0.02):
    """Nearly the same query in every row of a kv head's group, and its direction."""
    base = torch.randn(w.kv_heads, w.dim, generator=w.g, device="cuda")
    base = base / base.norm(dim=-1, keepdim=True) * math.sqrt(w.dim)
    q = base.repeat_interleave(w.heads // w.kv_heads, 0)[None] * (1 + spread * torch.randn(w.rows, w.heads, w.dim, generator=w.g, device="cuda"))
    return q.to(w.dtype), base.double()


def check(w, q, mask="causal", window=0, tree=None):
    """Against float64, row by row.  With u and U half a step of F16 and of the output, w = p times V's
    scale, and over the positions that the row sees alone:
      the error of key i's p is a factor within d_i = T_i (dim + 8) 2^-24 + 2^-21, T_i = scale sum |q k_i|
        (dim roundings of partial sums, those of the exponent's argument, exp2 itself);
      the numerator's: sum_i w_i |code_i| (u + d_i), its sum in float32 taken into another d_i, and for a
        product w that is small in its unit, half of F16's smallest step, 2^-25 of the unit, or all of w;
      the denominator's: sum_i p_i d_i of |o|; the output's rounding U |o|, 2^-25 at least for F16."""
    cache, batch = w.handles(P)
    o, lse = torch.full((w.rows, w.heads, w.dim), 7.0, dtype=w.dtype, device="cuda"), torch.full((w.rows, w.heads), 7.0, device="cuda")
    P.paged_attend(cache, batch, q, o, mask=mask, window=window, tree=tree, lse=lse)
    assert P.paged_device_error() == 0
    group = w.heads // w.kv_heads
    u = UNIT[torch.float16]
    for s, (n, kv) in enumerate(w.lens):
        r = slice(int(w.q_start[s]), int(w.q_start[s]) + n)
        at = torch.arange(kv, device="cuda")
        vs = w.vs[w.pages[s][at // w.page].long(), :, at % w.page].double().abs().repeat_interleave(group, 1)     # [kv, heads]
        k, v = w.K[s].repeat_interleave(group, 1), w.V[s].repeat_interleave(group, 1)
        code = torch.where(vs[..., None] > 0, v.abs() / vs[..., None], 0.0)
        x = q[r].double()
        z = torch.einsum("ihd,phd->hip", x, k) / math.sqrt(w.dim)
        z = z.masked_fill(w.hidden(s, mask, window, tree)[None], -math.inf)
        p = torch.softmax(z, -1).nan_to_num(0.0)
        T = torch.einsum("ihd,phd->hip", x.abs(), k.abs()) / math.sqrt(w.dim)
        d = T * (w.dim + 8) * 2.0 ** -24 + 2.0 ** -21
        weight = p * vs.T[:, None]
        least = torch.minimum(weight, 2.0 ** -25 * UNIT_ABOVE_WEIGHT * weight.amax(-1, keepdim=True))
        want = torch.einsum("hip,phd->ihd", p, v)
        off = torch.einsum("hip,phd->ihd", weight * (u + 2 * d) + least, code)
        denominator = (p * d).sum(-1).T[..., None]
        tol = off + (denominator + UNIT[w.dtype]) * want.abs() + (2.0 ** -25 if w.dtype == torch.float16 else 1e-38)
        got = o[r].double()
        fits = want.abs() < 6e4 if w.dtype == torch.float16 else torch.ones_like(want, dtype=torch.bool)
        bad = ~((got - want).abs() <= tol) & fits
        assert not bad.any(), (s, int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got - want).abs() / tol)[fits].max()))
        wl, some = torch.logsumexp(z, -1).T, (p.sum(-1) > 0).T
        lerr = (lse[r].double() - wl).abs() / (2 * denominator[..., 0] + 2.0 ** -22 * wl.abs() + 1e-30)
        assert (lerr[some] <= 1).all(), float(lerr[some].max())


CODED = [("int8", "f16"), ("int8", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")]
#: new tokens, 4 query heads to a kv head: the streaming kernel, dealt items of one block, items of two blocks
ROWS = [3, 9, 50]


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("power", [12, 20, 40])
def test_large_k_scales_out_of_sight(fmt, dtype, dim, n, power):
    """A K row with a large scale behind a row's last position, in its tile, and one in its sight that
    is far from its direction.  (The last token's own, which it sees, stays where float32 scores are worth
    something.)"""
    w = World([(n, 210), (1, 70), (n, n)], fmt=fmt, dtype=dtype, dim=dim, seed=power + n)
    q, base = queries(w)
    for s, (m, kv) in enumerate(w.lens):
        f = torch.ones(kv, w.kv_heads, device="cuda")
        if m > 1:
            f[-1] = 2.0 ** min(power, 20)
            rescale(w, s, "k", f)
        if kv > 100:
            put_keys(w, s, [5], base, [-(2.0 ** power)])
    check(w, q)


def clamp_power(w, power):
    """F16 outputs reach 65,504 only: what lies so far above the others lies as far below 2^12."""
    return 2.0 ** (min(0, 12 - power) if w.dtype == torch.float16 else 0)


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("power", [14, 20, 30, 100])
@pytest.mark.parametrize("where", ["first", "middle"])
def test_large_v_scales_without_weight(fmt, dtype, dim, n, power, where):
    """Seen by every row, but with a score far below all others (e^-100)."""
    w = World([(n, 500), (1, 70), (n, n + 3)], fmt=fmt, dtype=dtype, dim=dim, seed=power + n)
    q, base = queries(w)
    for s, (m, kv) in enumerate(w.lens):
        at = 0 if where == "first" else kv // 2
        put_keys(w, s, [at], base, [-100.0])
        f = torch.ones(kv, w.kv_heads, device="cuda")
        f[at] = 2.0 ** power
        rescale(w, s, "v", f * clamp_power(w, power if power < 100 else 0))
    check(w, q)


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("power", [14, 20, 30, 100])
def test_large_v_scales_out_of_sight(fmt, dtype, dim, n, power):
    """The batch's last tokens', which the ones before them do not see, in their tile."""
    w = World([(n, 500), (n, 130), (n, n)], fmt=fmt, dtype=dtype, dim=dim, seed=power + n)
    q, _ = queries(w)
    for s, (m, kv) in enumerate(w.lens):
        f = torch.ones(kv, w.kv_heads, device="cuda")
        f[-1] = 2.0 ** power
        f[-2, 0] = 2.0 ** -power
        rescale(w, s, "v", f)
    check(w, q)
    tree = torch.zeros(w.rows, dtype=torch.int64, device="cuda")
    for s, (m, _) in enumerate(w.lens):
        for i in range(m):
            tree[int(w.q_start[s]) + i] = (1 << i) | (1 << max(0, i - 2))
    check(w, q, "tree", tree=tree)


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("window", [0, 200])
def test_v_scales_of_all_sizes(fmt, dtype, n, window):
    """Forty powers of two up and down at random: what is largest counts most, the rest is small beside it."""
    w = World([(n, 700), (1, 300), (n, n)], fmt=fmt, dtype=dtype, seed=n)
    q, _ = queries(w, 1.0)
    for s, (m, kv) in enumerate(w.lens):
        up = torch.empty(kv, w.kv_heads, device="cuda").uniform_(-40, 40 if dtype == "bf16" else 10, generator=w.g)
        rescale(w, s, "v", torch.exp2(up))
    check(w, q, window=window)


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("rise,fall", [(0.3, 0.12), (0.3, -0.1), (-0.3, -0.12), (-0.3, 0.1), (1.5, 0.2)])
def test_weights_that_move(fmt, dtype, dim, n, rise, fall):
    """Scores that rise or fall along the sequence while V scales fall or rise, so that the largest product
    and the largest scale are in different places, and either moves from tile to tile."""
    w = World([(n, 600), (n, 150)], fmt=fmt, dtype=dtype, dim=dim, seed=5 + n)
    q, base = queries(w, 0.001)
    for s, (m, kv) in enumerate(w.lens):
        p = torch.arange(kv, device="cuda")
        score = rise * (p - kv)                       # natural units
        put_keys(w, s, p, base, score)
        up = -fall * p
        if dtype == "f16":                            # the largest near 1
            up = up - up.max()
        rescale(w, s, "v", torch.exp2(up)[:, None].expand(kv, w.kv_heads))
    check(w, q)


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("n", ROWS)
def test_v_rows_of_zeros_among_others(fmt, dtype, n):
    """Scales of 0 (rows below 1e-30) with nearly all the weight, and negative ones."""
    w = World([(n, 300), (1, 40)], fmt=fmt, dtype=dtype, seed=n)
    q, base = queries(w)
    for s, (m, kv) in enumerate(w.lens):
        f = torch.ones(kv, w.kv_heads, device="cuda")
        f[kv // 2::3] *= -1
        rescale(w, s, "v", f)
        zero = [0, kv // 3]
        put_keys(w, s, zero, base, [12.0, 12.0])
        page = w.pages[s][torch.tensor(zero, device="cuda") // w.page].long()
        w.vs[page, :, torch.tensor(zero, device="cuda") % w.page] = 0.0
        w.V[s][zero] = 0.0
    check(w, q)


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("block", [64, 128, 256])
@pytest.mark.parametrize("first", [0, 1])
def test_v_scales_by_the_tile(fmt, dtype, n, block, first):
    """Whole tiles of scales 2^20 above the others', with a 2^-24th of their weight: neither kind has far
    scales among its own, and both count."""
    w = World([(n, 1100), (1, 600)], fmt=fmt, dtype=dtype, seed=block + n)
    q, base = queries(w, 0.001)
    for s, (m, kv) in enumerate(w.lens):
        p = torch.arange(kv, device="cuda")
        large = p // block % 2 == first
        put_keys(w, s, p, base, torch.where(large, -24 * math.log(2.0), 0.1))
        up = torch.where(large, 20.0, 0.0) - (12.0 if dtype == "f16" else 0.0)
        rescale(w, s, "v", torch.exp2(up)[:, None].expand(kv, w.kv_heads))
    check(w, q)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("heavy", [3, 70, 200, 599])
@pytest.mark.parametrize("some", [39, 130, 411])
def test_a_row_of_zeros_with_all_the_weight(fmt, n, heavy, some):
    """One key has all the weight and a V row of zeros, another, e^-70 of it, all that comes out (as bf16
    values of some 1e-31), and zeros among the rest make every tile one of scales far apart."""
    w = World([(n, 650), (n, n + 620)], fmt=fmt, dtype="bf16", seed=heavy + some)
    q, base = queries(w, 0.001)
    for s, (m, kv) in enumerate(w.lens):
        p = torch.arange(kv - m, device="cuda")
        put_keys(w, s, p, base, torch.where(p == heavy, 70.0, torch.where(p == some, 0.0, -45.0)))
        put_keys(w, s, torch.arange(kv - m, kv, device="cuda"), base, torch.full((m,), -50.0))
        zero = torch.cat([torch.tensor([heavy], device="cuda"), torch.arange(81, kv - m, 17, device="cuda")])
        zero = zero[zero != some]
        w.vs[w.pages[s][zero // w.page].long(), :, zero % w.page] = 0.0
        w.V[s][zero] = 0.0
    check(w, q)
