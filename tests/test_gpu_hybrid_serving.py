"""The verifying model's two token mixers together, as a serving loop has them: one prompt's pages and recurrent state,
samples that branch from it, drafted blocks verified by paged_attend_shared and delta_rule, and a rejected tail taken
back in both -- in the cache by its length, in the recurrent layer by the slot behind the last accepted token."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from speculative_decoding_draft_kv_gb300 import paged as P
from tests.delta_oracle import UNIT
from tests.paged_oracle import norm_rope

pytestmark = pytest.mark.gpu

HEADS, KV, DIM = 8, 2, 128            # of the attention layer
DH, DK_HEADS, DK, DV = 8, 4, 128, 128  # of the recurrent layer
PAGE, EPS = 16, 1e-6


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Rows:
    """Random rows of one step, all tensors slices of two projections."""

    def __init__(self, g, n, dtype):
        def randn(*shape):
            return torch.randn(shape, device="cuda", generator=g)
        qkv = randn(n, HEADS + 2 * KV, DIM).to(dtype)
        self.q, self.k, self.v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        wide = randn(n, 2 * DK_HEADS * DK + DH * DV).to(dtype)
        self.dq, self.dk = wide[:, :DK_HEADS * DK].view(n, DK_HEADS, DK), wide[:, DK_HEADS * DK:2 * DK_HEADS * DK].view(n, DK_HEADS, DK)
        self.dv = wide[:, 2 * DK_HEADS * DK:].view(n, DH, DV)
        self.g, self.beta = -0.05 * torch.exp(randn(n, DH)), torch.sigmoid(randn(n, DH))
        self.n = n


class Recurrent:
    """One sequence's state in float64, and the bound of what a kernel's may be off (see delta_oracle)."""

    def __init__(self, state=None, off=0.0):
        self.S = torch.zeros(DH, DV, DK, dtype=torch.float64, device="cuda") if state is None else state.clone()
        self.off = off

    def token(self, r, i):
        q, k = (x[i].double().repeat_interleave(DH // DK_HEADS, 0) for x in (r.dq, r.dk))
        q, k = (x / (x.square().sum(-1, keepdim=True) + EPS).sqrt() for x in (q, k))
        q = q / math.sqrt(DK)
        v, a = r.dv[i].double(), torch.exp(r.g[i].double())[:, None, None]
        unit = 2.0 ** -20 * (torch.linalg.matrix_norm(self.S) + v.norm(dim=-1)).max()
        S = self.S * a
        u = r.beta[i].double()[:, None] * (v - (S @ k[..., None])[..., 0])
        self.S = S + u[..., None] * k[:, None]
        self.off = torch.sqrt(self.off ** 2 + (2 * unit) ** 2) if torch.is_tensor(self.off) else 2 * unit
        o = (self.S @ q[..., None])[..., 0]
        ql = q.norm(dim=-1)[:, None]
        return o, UNIT[r.dq.dtype] * o.abs() + (4 * (self.off + unit) + 2.0 ** -11 * self.S.norm(dim=-1)) * ql + 2.0 ** -25


@pytest.mark.parametrize("dtype,fmt", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.int8)])
@pytest.mark.parametrize("graph", [False, True])
def test_branches_of_a_prompt(dtype, fmt, graph):
    g = torch.Generator(device="cuda").manual_seed(3)
    n_seq, block, length, steps = 6, 5, 213, 4
    rope = P.PagedRope(DIM, 1e6)
    w = 1 + 0.1 * torch.randn(DIM, device="cuda", generator=g)
    coded = fmt == torch.int8
    n_pages, per = 64, 4
    pools = [torch.zeros(n_pages, KV, PAGE, DIM, dtype=fmt, device="cuda") for _ in range(2)]
    scales = [torch.zeros(n_pages, KV, PAGE, device="cuda") if coded else None for _ in range(2)]
    cache = P.PagedCache(*pools, *scales)
    shared = -(-length // PAGE)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    prompt_pages, own_pages = order[:shared][None].contiguous(), order[shared:shared + n_seq * per].view(n_seq, per).contiguous()

    def cached(i, kv, table):
        """Rows of a sequence as the cache has them [kv, KV, DIM], float64."""
        p = torch.arange(kv, device="cuda")
        ids, slot = table[i][p // PAGE].long(), p % PAGE
        x = [pool[ids, :, slot].double() for pool in pools]
        return [y * s[ids, :, slot].double()[..., None] for y, s in zip(x, scales)] if coded else x

    # states: slot 0 the prompt's, then one for every row of a step, twice over
    rows = n_seq * block
    state = torch.full((1 + 2 * rows, DH, DV, DK), math.nan, device="cuda")
    states = D.DeltaState(state)

    # the prompt, once for all: its pages and its state
    r = Rows(g, length, dtype)
    q_rot = torch.empty_like(r.q)
    P.paged_append(cache, P.PagedBatch(ints([0, length]), ints([length]), prompt_pages, length), r.k, r.v, rope=rope, eps=EPS, k_norm=w,
                   q=r.q, q_norm=w, q_out=q_rot)
    o = torch.empty(length, DH, DV, dtype=dtype, device="cuda")
    D.delta_rule(states, D.DeltaBatch(ints([0, length]), ints([-1]), ints([0]), length), r.dq, r.dk, r.dv, r.g, r.beta, o, eps=EPS)
    base = Recurrent()
    for i in range(length):
        want, tol = base.token(r, i)
        assert ((o[i].double() - want).abs() <= tol).all(), i
    assert (torch.linalg.matrix_norm(state[0].double() - base.S) <= 4 * base.off).all()

    # a step of all branches, and what a captured one has to follow
    q_start = ints([i * block for i in range(n_seq + 1)])
    kv_len, positions = ints([0] * n_seq), ints([0] * rows)
    slot_in, save = ints([0] * n_seq), ints([0] * rows)
    none = ints([-1] * n_seq)
    batch = P.PagedBatch(q_start, kv_len, own_pages, block)
    prefix = P.PagedBatch(ints([0, rows]), ints([length]), prompt_pages, rows)
    recurrent = D.DeltaBatch(q_start, slot_in, none, block, save=save)
    now = Rows(g, rows, dtype)
    q_rot, att = torch.empty_like(now.q), torch.empty(rows, HEADS, DIM, dtype=dtype, device="cuda")
    rec = torch.empty(rows, DH, DV, dtype=dtype, device="cuda")
    ws = torch.empty(P.paged_attend_shared_workspace(cache, batch, prefix, rows, HEADS), dtype=torch.uint8, device="cuda")

    def step():
        P.paged_append(cache, batch, now.k, now.v, rope=rope, eps=EPS, k_norm=w, q=now.q, q_norm=w, q_out=q_rot, positions=positions)
        P.paged_attend_shared(cache, batch, prefix, q_rot, att, workspace=ws)
        D.delta_rule(states, recurrent, now.dq, now.dk, now.dv, now.g, now.beta, rec, eps=EPS)

    taken = [0] * n_seq                              # own tokens that stand
    branches = [Recurrent(base.S, base.off) for _ in range(n_seq)]
    kept = [0] * n_seq                               # their states' slots
    replay = None
    for t in range(steps):
        fresh = Rows(g, rows, dtype)
        for a in ("q", "k", "v", "dq", "dk", "dv", "g", "beta"):
            getattr(now, a).copy_(getattr(fresh, a))
        kv_len.copy_(ints([x + block for x in taken]))
        positions.copy_(ints([length + x + i for x in taken for i in range(block)]))
        slot_in.copy_(ints(kept))
        mine = 1 + (t % 2) * rows
        save.copy_(ints([mine + i for i in range(rows)]))
        if graph and t == 1:                         # (the first step ran by itself: everything is set up)
            torch.cuda.synchronize()
            replay = torch.cuda.CUDAGraph()
            with torch.cuda.graph(replay):
                step()
        replay.replay() if replay else step()
        assert P.paged_device_error() == 0 and D.delta_device_error() == 0
        turned = norm_rope(now.q, positions, w, EPS, rope)
        assert ((q_rot.double() - turned).abs() <= 2 * UNIT[dtype] * turned.abs() + 2e-5).all()
        pk, pv = cached(0, length, prompt_pages)
        for s in range(n_seq):
            kv = taken[s] + block
            ok, ov = cached(s, kv, own_pages)
            k, v = torch.cat([pk, ok]), torch.cat([pv, ov])
            for i in range(block):
                row, seen = s * block + i, length + taken[s] + i + 1
                q = q_rot[row].double()
                for h in range(HEADS):
                    z = k[:seen, h // (HEADS // KV)] @ q[h] / math.sqrt(DIM)
                    p = torch.softmax(z, 0)
                    want = p @ v[:seen, h // (HEADS // KV)]
                    size = p @ v[:seen, h // (HEADS // KV)].abs()
                    # (probabilities and outputs rounded, scores' sums: see paged_oracle)
                    tol = 2 * UNIT[dtype] * (size + want.abs()) + 1e-5 * size + 1e-5
                    assert ((att[row, h].double() - want).abs() <= tol).all(), (t, s, i, h)
            accepted = int(torch.randint(0, block + 1, (1,), generator=g, device="cuda"))
            x, goes_on = branches[s], branches[s]
            for i in range(block):
                x = Recurrent(x.S, x.off)
                want, tol = x.token(now, s * block + i)
                assert ((rec[s * block + i].double() - want).abs() <= tol).all(), (t, s, i)
                assert (torch.linalg.matrix_norm(state[mine + s * block + i].double() - x.S) <= 4 * x.off).all()
                if i + 1 == accepted:
                    goes_on = x
            if accepted:
                kept[s] = mine + s * block + accepted - 1
            branches[s] = goes_on
            taken[s] += accepted
            # a slot that the next step writes may not be one that it reads: a branch that stood still moves its state
            if not accepted and kept[s] and t + 1 < steps:
                other = 1 + (t % 2) * rows + s * block
                state[other].copy_(state[kept[s]])
                kept[s] = other
