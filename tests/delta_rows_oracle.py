"""The gated delta rule in float64 with bounds for each row of a state (value element) by itself: rows never meet, so what one
holds may not cost another its precision."""

import torch

from tests.delta_oracle import UNIT


def want_rows(w, max_q=None, normalise=True, eps=1e-6, scale=0.0):
    """(o, bound of o, {slot: (state, bound of its rows' norms [heads, dim_v])}) of a DeltaWorld before the call is made.

    Of one row S (a vector over the key's elements), with |k| <= 1 and 0 <= beta <= 2: a step S -> a S (I - beta k k^T) + beta v k^T
    lengthens no error, so what a step rounds off is carried on times a = exp(g) at most.
      A step rounds the sum S k (dim_k products of random signs, 2^-24 sqrt(dim_k) = 2^-20.5 of |S| for 128), or takes operands of
    22 bits (2^-22 of |S| and of |u|, each a few times), all of the decayed row and v:
        E^2 <- (a E)^2 + (2^-20 (|a S| + |v|))^2,
    independent roundings whose squares add; four times E is allowed.
      What is the same each time a key comes again (its norm's rounding, the cut-off ends of sums) is a factor of S k of at most
    1 + 2^-20, and adds as it is: F <- a F + 2^-20 beta |a S k|.
      Sequences of more than 8 tokens of a batch whose max_q is above 12 are worked on 32 tokens at a time, by u = T r with
    r_j = beta_j (v_j - exp(G_j) S0 k_j), S0 the row in front of the chunk and T the inverse of a unit triangular matrix with
    entries of at most beta below the diagonal, each off by 2^-19 max(beta^3, beta / 8) (31 products of entries up to beta and beta,
    rounded by 2^-24 of it, sqrt(32) of that, and again sqrt(32) beta of it in the rows behind; as an operand 2^-22 beta):
        E^2 <- E^2 + (2^-19 max(beta^3, beta / 8))^2 sum_{j <= i} r_j^2.
    r is an operand in one unit for the chunk's 32 tokens: its two F16 parts reach down to 2^-25 where the largest is 2^5 or more, so each
    r_j is off by 2^-30 of the largest, whichever token that is, and u by 2^-30 beta sqrt(32) of it, below 2^-26:
        E^2 <- E^2 + (2^-26 max_j r_j)^2.
    Decays and states end at float32's smallest step, 2^-149 (halves of it where a product or an exponential is rounded there): a token
    adds that of each element, and of exp(g) or exp(G) times what it multiplies, (2^-149 (2 sqrt(dim_k) + |S| + |S0|))^2.
      An output is off by |q| times the state's error, by its own sum (2^-20 (|a S| + |v|) |q|) and by its rounding (F16's
    smallest step is 2^-24, bf16's 2^-133).  In chunks, bf16 outputs take S0 as one F16, off by 2^-11 of each element: 2^-11 exp(G) |S0| |q|."""
    max_q = max([*w.lens, 0]) if max_q is None else max_q
    pool = w.pool.double().clone()
    group = w.heads // w.heads_k
    out = torch.zeros(w.total, w.heads, w.dim_v, dtype=torch.float64, device="cuda")
    tol, slots = torch.zeros_like(out), {}
    q, k = (x[:w.total].double().repeat_interleave(group, 1) for x in (w.q, w.k))
    if normalise:
        q, k = (x / (x.square().sum(-1, keepdim=True) + eps).sqrt() for x in (q, k))
    q = q * (scale or w.dim_k ** -0.5)
    v, beta = w.v[:w.total].double(), w.beta[:w.total].double()
    decay = w.decay[:w.total].double().clamp(min=-1e4)
    for s, n in enumerate(w.lens):
        S = pool[w.slot_in[s]].clone() if w.slot_in[s] >= 0 else torch.zeros_like(pool[0])
        E, F = torch.zeros(2, w.heads, w.dim_v, dtype=torch.float64, device="cuda")
        long = n > 8 and max_q > 12 and w.save is None
        for i in range(n):
            r = w.starts[s] + i
            if long and i % 32 == 0:
                c = slice(r, w.starts[s] + min(n, i + 32))
                S0 = S.norm(dim=-1)
                G = decay[c].cumsum(0).exp()                                                         # [tokens, heads]
                sk = torch.einsum("hvk,thk->thv", S, k[c]).abs() * G[..., None]
                R = beta[c].abs()[..., None] * (v[c].abs() + sk)
                most, sums = R.amax(0), R.square().cumsum(0)
            a, b = decay[r].exp()[:, None], beta[r].abs()[:, None]
            least = 2.0 ** -149 * (2 * w.dim_k ** 0.5 + S.norm(dim=-1) + (S0 if long else 0.0))
            S = S * a[..., None]
            unit = 2.0 ** -20 * (S.norm(dim=-1) + v[r].abs())
            sk = (S @ k[r][..., None])[..., 0]
            F = a * F + 2.0 ** -20 * b * sk.abs()
            S = S + (beta[r][:, None] * (v[r] - sk))[..., None] * k[r][:, None]
            E = (a * E) ** 2 + unit ** 2 + least ** 2
            if long:
                E = E + (2.0 ** -19 * torch.maximum(b ** 3, b / 8)) ** 2 * sums[i % 32] + (2.0 ** -26 * most) ** 2
            E = E.sqrt()
            out[r] = (S @ q[r][..., None])[..., 0]
            ql = q[r].norm(dim=-1)[:, None]
            tol[r] = UNIT[w.dtype] * out[r].abs() + (4 * (E + unit) + F) * ql
            tol[r] += 2.0 ** -25 if w.dtype == torch.float16 else 2.0 ** -134
            if long and w.dtype == torch.bfloat16:
                tol[r] += 2.0 ** -11 * G[i % 32][:, None] * S0 * ql
            if w.save is not None and 0 <= w.save[r] < w.n_slots:
                slots[w.save[r]] = (S.clone(), 4 * E + F)
        if 0 <= w.slot_out[s] < w.n_slots:
            slots[w.slot_out[s]] = (S, 4 * E + F)
    return out, tol, slots


def check_rows(w, D, max_q=None, **kw):
    """Runs the operator and holds every value element to want_rows()."""
    out, tol, slots = want_rows(w, max_q, **kw)
    state, batch = w.handles(D, max_q)
    o = torch.empty(w.rows, w.heads, w.dim_v, dtype=w.dtype, device="cuda")
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o, **kw)
    assert D.delta_device_error() == 0
    off = (o[:w.total].double() - out).abs()
    far = ~(off <= tol)
    assert not far.any(), ("o", int(far.sum()), float((off / tol).nan_to_num(9e9).max()), far.nonzero()[:4].tolist())
    for slot, (S, bound) in slots.items():
        off = (w.pool[slot].double() - S).norm(dim=-1)
        far = ~(off <= bound)
        assert not far.any(), ("slot", slot, int(far.sum()), float((off / bound).nan_to_num(9e9).max()), far.nonzero()[:4].tolist())
