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
UNIT_ABOVE_WEIGHT = 2.0 ** 8


def rescale(w, s, which, factor):
    """The scales of sequence s's K or V rows times factor [kv, kv_heads]."""
    pool, true = (w.ks, w.K) if which == "k" else (w.vs, w.V)
    p = torch.arange(w.lens[s][1], device="cuda")
    page, slot = w.pages[s][p // w.page].long(), p % w.page
    old = pool[page, :, slot]
    new = (old * factor).float()
    pool[page, :, slot] = new
    true[s] = true[s] * (new.double() / old.double())[..., None]


def put_key(w, s, positions, direction, length):
    """K rows of some positions along direction [kv_heads, dim], of scale-free length `length`."""
    x = direction / direction.abs().amax(-1, keepdim=True) * 100
    codes = x.round() if w.store == torch.int8 else x.to(w.store).float()
    for p in positions:
        page, slot = int(w.pages[s, p // w.page]), p % w.page
        size = codes.double().square().sum(-1).sqrt()
        scale = (length[p] / size).float()
        w.k.view(torch.uint8)[page, :, slot] = codes.to(w.store).view(torch.uint8)
        w.ks[page, :, slot] = scale
        w.K[s][p] = codes.double() * scale.double()[:, None]


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
        code = v.abs() / vs[..., None]
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
WIDE = [9, 50]              # new tokens, 4 query heads to a kv head: dealt items of one block, items of two


@pytest.mark.parametrize("fmt,dtype", CODED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [3] + WIDE)
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
            put_key(w, s, [5], -base, {5: 2.0 ** power})
    check(w, q)
