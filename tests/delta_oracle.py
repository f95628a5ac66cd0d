"""The gated delta rule in float64, token by token, with the bounds that a kernel's results are held to."""

import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}     # half a step


class DeltaWorld:
    """A batch with its pool: ``lens`` are the sequences' new tokens; every slot that nothing reads is full of NaN."""

    def __init__(self, lens, heads=4, heads_k=2, dim_k=128, dim_v=128, dtype=torch.bfloat16, seed=0, spare_rows=0,
                 slots=None, spread=1.0, rate=0.1):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.heads, self.heads_k, self.dim_k, self.dim_v, self.dtype = lens, heads, heads_k, dim_k, dim_v, dtype
        n, self.total = len(lens), sum(lens)
        self.rows = self.total + spare_rows

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.q, self.k = (randn(self.rows, heads_k, dim_k).to(dtype) for _ in range(2))
        self.v = (randn(self.rows, heads, dim_v) * spread).to(dtype)
        self.decay = -rate * torch.exp(randn(self.rows, heads))
        self.beta = torch.sigmoid(randn(self.rows, heads))
        for x in (self.q, self.k, self.v, self.decay, self.beta):
            x[self.total:] = float("nan")
        self.starts = [sum(lens[:i]) for i in range(n + 1)]
        self.q_start = self.ints(self.starts)
        # slots 0 .. n-1 are read, n .. 2n-1 written
        self.n_slots = slots or 2 * n + 3
        self.pool = torch.full((self.n_slots, heads, dim_v, dim_k), float("nan"), device="cuda")
        self.pool[:n] = randn(n, heads, dim_v, dim_k) * 0.3 * spread
        self.slot_in = list(range(n))
        self.slot_out = list(range(n, 2 * n))
        self.save = None

    @staticmethod
    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def handles(self, D, max_q=None):
        save = None if self.save is None else self.ints(self.save)
        return D.DeltaState(self.pool), D.DeltaBatch(self.q_start, self.ints(self.slot_in), self.ints(self.slot_out),
                                                     max([*self.lens, 0]) if max_q is None else max_q, save=save)

    def want(self, normalise=True, eps=1e-6, scale=0.0):
        """(o, bound of o, {slot: (state, bound of its norm by head)}) before the call is made.

        With |k| = 1 and 0 <= beta <= 2 a step S -> exp(g) S (I - beta k k^T) lengthens no row of S, so what a step
        rounds off is only ever carried on, times exp(g).  A step rounds sums of dim_k products (of random signs:
        2^-24 sqrt(dim_k) = 2^-20.5 of |S| for 128) or operands of 22 bits (2^-22 of |S| and of |u|, each a few
        times), all relative to |S|_F + |v|.  These roundings are independent, so their squares add:
            E^2 <- exp(2 g) E^2 + (2^-20 (|S|_F + |v|))^2,
        and four times that is allowed.  What is not independent is the norm of a key that comes again: its rounding
        (2^-23) and the cut-off ends of the sums that k . k and S k are (16 of up to 2^-24 each, always towards
        zero: 2^-21 on average) are the same each time, and change S k by a factor, so these errors add as they are:
            F <- exp(g) F + 2^-20 beta |S k|.
        A sequence of more than 8 tokens is worked on 32 at a time, through the inverse T of I + L, L_ij = beta_i exp(..)
        k_i . k_j: its updates are u = T r, r_j = beta_j (v_j - exp(..) S k_j).  T_ij = -beta_i k_i . (what a key passes
        through between) k_j, at most beta_i.  Substitution gets a row of T from those above it: 31 products of L and
        T, each rounded (2^-24 beta_i beta, together sqrt(32) of it), and what is off there comes on multiplied by
        a row of T again (sqrt(32) beta): 2^-24 32 beta^3 = 2^-19 beta^3 an entry; as an operand it has 22 bits, 2^-22 beta.
        Entries and tokens are independent, so a token adds
            E^2 <- E^2 + (2^-19 max(beta^3, beta / 8))^2 sum of |r_j|^2 over the chunk's tokens up to it.
        (It takes keys alike and beta of 2 for that to count beside the rest.)
        An output is off by |q| times the state's error and by its own
        rounding, and q . S's sum like k . S's; over many tokens bf16 outputs take S as one F16, half a step (2^-11) of
        each product, together at most 2^-11 |S_row| |q|."""
        n = len(self.lens)
        pool = self.pool.double().clone()
        out = torch.zeros(self.total, self.heads, self.dim_v, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        slots = {}
        group = self.heads // self.heads_k
        q, k = (x[:self.total].double().repeat_interleave(group, 1) for x in (self.q, self.k))
        if normalise:
            q, k = (x / (x.square().sum(-1, keepdim=True) + eps).sqrt() for x in (q, k))
        q = q * (scale or self.dim_k ** -0.5)
        for s in range(n):
            at = self.slot_in[s]
            S = pool[at].clone() if at >= 0 else torch.zeros_like(pool[0])
            E, F = torch.zeros(2, self.heads, dtype=torch.float64, device="cuda")
            long = self.lens[s] > 8 and self.save is None
            for r in range(self.starts[s], self.starts[s + 1]):
                if (r - self.starts[s]) % 32 == 0:
                    S0, rr = S, torch.zeros_like(E)
                a = torch.exp(self.decay[r].double())
                unit = 2.0 ** -20 * (torch.linalg.matrix_norm(S) + self.v[r].double().norm(dim=-1))
                S = S * a[:, None, None]
                sk = (S @ k[r][..., None])[..., 0]
                u = self.beta[r].double()[:, None] * (self.v[r].double() - sk)
                F = a * F + 2.0 ** -20 * self.beta[r].double() * sk.norm(dim=-1)
                S = S + u[..., None] * k[r][:, None]
                b = self.beta[r].double().abs()
                rr = rr + (b * (self.v[r].double().norm(dim=-1) + (S0 @ k[r][..., None])[..., 0].norm(dim=-1))) ** 2
                solve = 2.0 ** -19 * torch.maximum(b ** 3, b / 8) if long else torch.zeros_like(E)
                E = torch.sqrt((a * E) ** 2 + unit ** 2 + solve ** 2 * rr)
                out[r] = (S @ q[r][..., None])[..., 0]
                tol[r] = UNIT[self.dtype] * out[r].abs() + ((4 * (E + unit) + F) * q[r].norm(dim=-1))[:, None] + (
                    2.0 ** -11 * S.norm(dim=-1) * q[r].norm(dim=-1)[:, None] if self.dtype == torch.bfloat16 else 0.0) + (
                    2.0 ** -25 if self.dtype == torch.float16 else 0.0)
                if self.save is not None and 0 <= self.save[r] < self.n_slots:
                    slots[self.save[r]] = (S.clone(), 4 * E + F)
            if 0 <= self.slot_out[s] < self.n_slots:
                slots[self.slot_out[s]] = (S, 4 * E + F)
        return out, tol, slots

    def check(self, D, normalise=True, eps=1e-6, scale=0.0, o=None, max_q=None, errors=0, run=None):
        """Runs the operator and holds it to want(): outputs, slots, and what must stay as it was."""
        out, tol, slots = self.want(normalise, eps, scale)
        before = self.pool.clone()
        state, batch = self.handles(D, max_q)
        if o is None:
            o = torch.empty(self.rows, self.heads, self.dim_v, dtype=self.dtype, device="cuda")
        o.fill_(7.0)
        call = lambda: D.delta_rule(state, batch, self.q, self.k, self.v, self.decay, self.beta, o,     # noqa: E731
                                    normalise=normalise, eps=eps, scale=scale)
        run(call) if run else call()
        assert D.delta_device_error() == errors
        off = (o[:self.total].double() - out).abs()
        assert (off <= tol).all(), ("o", float((off / tol).nan_to_num(9e9).max()), (~(off <= tol)).nonzero()[:4].tolist())
        assert (o[self.total:] == 7.0).all(), "rows behind the batch"
        for slot, (S, bound) in slots.items():
            far = torch.linalg.matrix_norm(self.pool[slot].double() - S)
            assert (far <= bound).all(), ("slot", slot, (far / bound).tolist())
        for slot in range(self.n_slots):
            if slot not in slots:
                assert torch.equal(self.pool[slot].view(torch.int32), before[slot].view(torch.int32)), slot
        return o
