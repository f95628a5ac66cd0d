"""Float64 forms of the paged operators, and worlds to try them in: pools full of what must not
matter (NaN, or NaN scales over arbitrary codes) with the sequences' rows scattered over them."""

import math

import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
FORMATS = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}    # half a step


def norm_rope(x, positions, w, eps, rope):
    """x [rows, heads, dim] -> float64."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    if rope is None:
        return x
    r = rope.args.rotary_dim
    a = positions.double()[:, None, None] * torch.tensor(rope.inv_freq, dtype=torch.float64, device=x.device)
    c, s = torch.cos(a) * rope.magnitude, torch.sin(a) * rope.magnitude
    y = x.clone()
    one, two = (slice(0, r // 2), slice(r // 2, r)) if rope.args.layout == 0 else (slice(0, r, 2), slice(1, r, 2))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., one] * s + x[..., two] * c
    return y


class World:
    """A batch of sequences over pages: ``lens`` holds (new tokens, cached tokens with them)."""

    def __init__(self, lens, page=16, heads=8, kv_heads=2, dim=128, fmt="f16", dtype="f16", seed=0, order="hnd",
                 spare_rows=0, fill=True, poison=True, spread=1.0):
        self.lens, self.page, self.heads, self.kv_heads, self.dim = lens, page, heads, kv_heads, dim
        self.fmt, self.store, self.dtype = fmt, FORMATS[fmt], FORMATS[dtype]
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        used = [-(-kv // page) for _, kv in lens]
        self.n_pages = sum(used) + 3
        ids = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        self.max_pages = max(used + [1])
        self.pages = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32, device="cuda")
        at = 0
        for s, u in enumerate(used):
            self.pages[s, :u] = ids[at:at + u]
            at += u
        self.q_start = torch.tensor([sum(n for n, _ in lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                                    device="cuda")
        self.kv_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
        self.total = int(self.q_start[-1])
        self.rows = self.total + spare_rows
        shape = (self.n_pages, kv_heads, page, dim)

        def pool():
            if order == "hnd":
                x = torch.empty(shape, dtype=torch.float32, device="cuda")
            else:                        # [page, token, head, dim]
                x = torch.empty((self.n_pages, page, kv_heads, dim), dtype=torch.float32, device="cuda").transpose(1, 2)
            if self.store in TOP:
                x.copy_(torch.randint(-100, 100, shape, generator=g, device="cuda"))
            else:
                x.fill_(math.nan if poison else 0.0)
            y = torch.empty_strided(shape, x.stride(), dtype=self.store, device="cuda")
            return y.copy_(x)

        self.k, self.v = pool(), pool()
        self.ks = self.vs = None
        if self.store in TOP:
            self.ks, self.vs = (torch.full(shape[:3], math.nan if poison else 0.0, device="cuda") for _ in range(2))
        # the true rows of each sequence [kv, kv_heads, dim], float64
        self.K, self.V = [], []
        for s, (_, kv) in enumerate(lens):
            for pool_, scale, keep in ((self.k, self.ks, self.K), (self.v, self.vs, self.V)):
                x = torch.randn(kv, kv_heads, dim, generator=g, device="cuda") * spread
                if not fill:
                    keep.append(x.double())
                    continue
                p = torch.arange(kv, device="cuda")
                page_id, slot = self.pages[s][p // page].long(), p % page
                if scale is None:
                    x = x.to(self.store)
                    pool_[page_id, :, slot] = x
                    keep.append(x.double())
                else:
                    codes = (x * TOP[self.store] / 4).clamp(-TOP[self.store], TOP[self.store])
                    codes = codes.round().to(self.store) if self.store == torch.int8 else codes.to(self.store)
                    sc = torch.exp(torch.randn(kv, kv_heads, generator=g, device="cuda")) * 4 / TOP[self.store]
                    pool_.view(torch.uint8)[page_id, :, slot] = codes.view(torch.uint8)
                    scale[page_id, :, slot] = sc
                    keep.append(codes.double() * sc.double()[..., None])

    def randn(self, heads, dtype=None, spread=1.0):
        return (torch.randn(self.rows, heads, self.dim, generator=self.g, device="cuda") * spread).to(dtype or self.dtype)

    def handles(self, P, max_q=None, max_kv=0):
        cache = P.PagedCache(self.k, self.v, self.ks, self.vs)
        batch = P.PagedBatch(self.q_start, self.kv_len, self.pages,
                             max(n for n, _ in self.lens) if max_q is None else max_q, max_kv)
        return cache, batch

    def hidden(self, s, mask, window, tree):
        """Truth values [n, kv]: what each new token does not see."""
        n, kv = self.lens[s]
        c = kv - n
        p = torch.arange(kv, device="cuda")[None]
        i = torch.arange(n, device="cuda")[:, None]
        if mask == "causal":
            h = p > c + i
            return h | (p <= c + i - window) if window else h
        h = (p < c - window).expand(n, kv) if window else torch.zeros(n, kv, dtype=torch.bool, device="cuda")
        if mask == "tree":
            q0 = int(self.q_start[s])
            word = tree[q0:q0 + n, None]
            h = torch.where(p >= c, ((word >> (p - c).clamp(0, 63)) & 1) == 0, h)
        return h

    def attend(self, q, mask="causal", window=0, tree=None, scale=None, wide=False):
        """(o, lse, tolerance of o, tolerance of lse) in float64, rows behind the batch left out.

        The tolerances are a kernel's that multiplies exactly, adds in float32 and rounds
        probabilities to its operand type (F16 over quantised pages) and the output to its own,
        u and U being half a step of the two:
          a score's error: dim roundings of partial sums, none above T = scale sum |q k|, and
            those of the exponent's argument, at most |score| log2(e) 2^-24 twice, which
            changes p by a factor within d = T (dim + 8) 2^-24, plus 2^-21 for exp2 itself;
          numerator u + d, denominator d, relative to A = sum softmax |v|; the sums over the
            keys, in float32, in runs of at most a few thousand terms: 2^-12 u more, kept in 2 d;
          F16's smallest step 2^-25 on each probability against at most the largest |v|;
          the output U |o|;
          wide (more than 32 query rows per kv head) over quantised pages, bf16: K and V rows are rounded
            to F16 first, by at most 2^-11 of each element, which moves a score by at most 2^-11 T
            and the numerator by 2^-11 A."""
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        o = torch.zeros(self.total, self.heads, self.dim, dtype=torch.float64, device="cuda")
        lse = torch.full((self.total, self.heads), -math.inf, dtype=torch.float64, device="cuda")
        tol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
        operand = torch.float16 if self.store in TOP else self.dtype
        group = self.heads // self.kv_heads
        for s, (n, kv) in enumerate(self.lens):
            if n == 0 or kv == 0:
                continue
            r = slice(int(self.q_start[s]), int(self.q_start[s]) + n)
            k = self.K[s].repeat_interleave(group, 1)
            v = self.V[s].repeat_interleave(group, 1)
            x = q[r].double()
            z = torch.einsum("ihd,phd->hip", x, k) * scale
            z = z.masked_fill(self.hidden(s, mask, window, tree)[None], -math.inf)
            lse[r] = torch.logsumexp(z, -1).T
            p = torch.softmax(z, -1).nan_to_num(0.0)
            o[r] = torch.einsum("hip,phd->ihd", p, v)
            T = (torch.einsum("ihd,phd->hip", x.abs(), k.abs()).amax(-1) * scale).T     # [n, heads]
            d = T * (self.dim + 8) * 2.0 ** -24 + 2.0 ** -21
            more = UNIT[torch.float16] if wide and self.store in TOP and self.dtype == torch.bfloat16 else 0.0
            d = d + more * T
            A = torch.einsum("hip,phd->ihd", p, v.abs())
            tiny = kv * 2.0 ** -25 * v.abs().amax() if operand == torch.float16 else 0.0
            tol[r] = (UNIT[operand] + more + 3 * d[..., None]) * A + UNIT[self.dtype] * o[r].abs() + tiny + 1e-30
            ltol[r] = 2 * d + 2.0 ** -22 * lse[r].abs().nan_to_num(posinf=0.0)
        return o, lse, tol, ltol
