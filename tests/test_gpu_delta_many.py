"""delta_rule over many tokens with many sequences and heads at once: the same bounds as elsewhere."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
HEADS = dict(heads=24, heads_k=12)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim_k", [64, 128])
@pytest.mark.parametrize("lens", [[9, 33], [32, 40], [130, 64], [200, 5, 0, 31]])
def test_types_sizes_and_lengths(dtype, dim_k, lens):
    DeltaWorld(lens, dim_k=dim_k, dtype=dtype, spare_rows=2, seed=sum(lens), **HEADS).check(D)


@pytest.mark.parametrize("n", [10, 31, 32, 33, 63, 64, 65, 95, 96, 97, 128, 161, 290])
def test_lengths(n):
    DeltaWorld([n, n + 1], dtype=F16, seed=n, **HEADS).check(D)


@pytest.mark.parametrize("heads,heads_k", [(40, 40), (20, 1), (41, 41), (64, 16)])
def test_head_groups(heads, heads_k):
    DeltaWorld([50, 12], heads=heads, heads_k=heads_k, seed=heads).check(D)


def test_more_heads_than_fit_at_once():
    DeltaWorld([70, 35, 100, 1, 40, 64, 9, 33, 77, 12, 20], heads=32, heads_k=16, seed=1).check(D)


def test_without_a_state_and_branches():
    w = DeltaWorld([60, 45, 30], seed=2, **HEADS)
    w.slot_in = [-1, 2, 2]
    w.pool[0] = math.nan
    w.check(D)


def test_in_place_and_not_kept():
    w = DeltaWorld([60, 90, 33], seed=3, **HEADS)
    w.slot_out = [0, -1, 2]
    w.check(D)


def test_strides():
    w = DeltaWorld([40, 70], heads=24, heads_k=12, seed=4)
    t = w.rows
    wide = torch.full((t, 2 * 12 * 128 + 24 * 128 + 64), math.nan, dtype=w.dtype, device="cuda")
    for name, at, heads in (("q", 0, 12), ("k", 12 * 128, 12), ("v", 24 * 128, 24)):
        part = wide[:, at:at + heads * 128].view(t, heads, 128)
        part.copy_(getattr(w, name))
        setattr(w, name, part)
    pool = torch.full((24, w.n_slots, 128, 128), math.nan, device="cuda").transpose(0, 1)
    pool.copy_(w.pool)
    w.pool = pool
    o = torch.full((t, 26, 136), 7.0, dtype=w.dtype, device="cuda")
    w.check(D, o=o[:, 1:25, :128])
    assert (o[:, 0] == 7).all() and (o[:, 25] == 7).all() and (o[:, :, 128:] == 7).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_the_same_key_again_and_again(dtype):
    for top in (1.0, 2.0):
        w = DeltaWorld([100, 40], dtype=dtype, seed=5, rate=1e-3, **HEADS)
        w.k[:] = w.k[:1].clone()
        w.beta[:] = top
        w.check(D)


def test_decays_from_none_to_all():
    n = 140
    w = DeltaWorld([n, 35], heads=24, heads_k=8, seed=6)
    w.decay[:n, 0] = 0.0
    w.decay[:n, 1] = -1e-6
    w.decay[:n, 2] = -30.0
    w.decay[n // 2, 3] = -math.inf
    w.decay[n // 3, 4] = -3.4e38
    w.decay[n // 3:n // 2 + 2, 5] = -1e4
    w.check(D)


@pytest.mark.parametrize("spread", [1e-6, 3e3, 1e12])
def test_far_magnitudes(spread):
    """Rows of a state, heads and tokens of all magnitudes."""
    w = DeltaWorld([66, 41], dtype=BF16, spread=spread, seed=7, **HEADS)
    w.v[:, 1] *= 2.0 ** -20
    w.pool[0, 2] *= 2.0 ** -20
    w.check(D)


@pytest.mark.parametrize("n", [40, 100])
def test_nan_and_infinities_stay_in_their_rows(n):
    w = DeltaWorld([n, n], heads=24, heads_k=24, seed=8)
    out, tol, slots = w.want()
    w.v[1, 0, 5] = math.nan
    w.v[3, 1, 9] = math.inf
    w.pool[0, 3, 7, 7] = math.inf
    state, batch = w.handles(D)
    o = torch.empty_like(w.v)
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
    assert D.delta_device_error() == 0
    bad = ~((o.double() - out).abs() <= tol)
    for head, row in ((0, 5), (1, 9), (3, 7)):
        assert bad[:n, head, row].any()
        bad[:n, head, row] = False
    assert not bad.any()
    for s in range(2):
        S, bound = slots[2 + s]
        far = (w.pool[2 + s].double() - S)
        if s == 0:
            for head, row in ((0, 5), (1, 9), (3, 7)):
                assert not torch.isfinite(far[head, row]).all()
                far[head, row] = 0
        assert (torch.linalg.matrix_norm(far) <= bound).all()


def test_broken_batches_are_left_alone():
    n = 50
    w = DeltaWorld([n] * 4, slots=20, seed=9, **HEADS)
    state, batch = w.handles(D)
    batch = D.DeltaBatch(w.ints([0, n, n - 1, n, 2 * n]), batch.tensors[1], batch.tensors[2], n)
    before, o = w.pool.clone(), torch.full_like(w.v, 7.0)
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
    assert D.delta_device_error() == D.DELTA_ERR_BATCH
    assert torch.equal(w.pool[5].view(torch.int32), before[5].view(torch.int32))
    for slot_in, slot_out, alone in (([0, 20, 2, 1 << 30], None, (1, 3)), (None, [4, 20, 6, 1 << 30], ())):
        w = DeltaWorld([n] * 4, slots=20, seed=9, **HEADS)
        w.slot_in, w.slot_out = slot_in or w.slot_in, slot_out or w.slot_out
        state, batch = w.handles(D)
        o = torch.full_like(w.v, 7.0)
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
        assert D.delta_device_error() == D.DELTA_ERR_SLOT
        for s in range(4):
            assert (o[s * n:s * n + n] == 7).all() == (s in alone)
        assert torch.isnan(w.pool[8:]).all()


def test_captured_and_replayed():
    n = 90
    w = DeltaWorld([n, n, n], seed=10, slots=12, **HEADS)
    state = D.DeltaState(w.pool)
    arrays = [w.q_start, w.ints(w.slot_in), w.ints(w.slot_out)]
    batch = D.DeltaBatch(*arrays, n)
    o = torch.empty_like(w.v)
    ws = torch.empty(D.delta_rule_workspace(state, batch, w.rows, w.heads_k), dtype=torch.uint8, device="cuda")
    call = lambda: D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o, workspace=ws)     # noqa: E731
    kept = w.pool.clone()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, slot_in, slot_out in (([n, n, n], [0, 1, 2], [3, 4, 5]), ([n - 1, 5, 40], [2, -1, 2], [6, 7, -1])):
        x = DeltaWorld(lens, seed=11 + lens[0], slots=12, spare_rows=3 * n - sum(lens), **HEADS)
        for a in ("q", "k", "v", "decay", "beta"):
            getattr(w, a).copy_(getattr(x, a))
        w.pool.copy_(kept)
        x.pool.copy_(kept)
        x.slot_in, x.slot_out = slot_in, slot_out
        for to, src in zip(arrays, (x.q_start, x.ints(slot_in), x.ints(slot_out))):
            to.copy_(src)
        out, tol, slots = x.want()
        o.fill_(7.0)
        ws.fill_(255)                                # nothing is kept between calls
        graph.replay()
        assert D.delta_device_error() == 0
        assert ((o[:x.total].double() - out).abs() <= tol).all() and (o[x.total:] == 7).all()
        for slot, (S, bound) in slots.items():
            assert (torch.linalg.matrix_norm(w.pool[slot].double() - S) <= bound).all()


def test_two_streams_at_once():
    worlds = [DeltaWorld([300, 50], seed=12, **HEADS), DeltaWorld([120, 33, 10], seed=13, **HEADS)]
    wants = [w.want() for w in worlds]
    jobs = []
    for w in worlds:
        jobs.append((*w.handles(D), torch.empty_like(w.v), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for w, (state, batch, o, st) in zip(worlds, jobs):
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o, stream=st)
    assert D.delta_device_error() == 0
    for w, (_, _, o, _), (out, tol, slots) in zip(worlds, jobs, wants):
        assert ((o.double() - out).abs() <= tol).all()
        for slot, (S, bound) in slots.items():
            assert (torch.linalg.matrix_norm(w.pool[slot].double() - S) <= bound).all()


def test_the_same_call_gives_the_same_bits():
    w = DeltaWorld([150, 60], seed=14, **HEADS)
    state, batch = w.handles(D)
    got = []
    for _ in range(3):
        o = torch.empty_like(w.v)
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
        got.append((o.view(torch.int16).clone(), w.pool[2:4].view(torch.int32).clone()))
    assert all(torch.equal(a, b) for x in got[1:] for a, b in zip(x, got[0]))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,heads", [([4000, 3900, 2400, 830, 3300, 1800, 240, 2700], 32), ([6000, 4000], 32), ([12000], 48)])
def test_long_sequences_give_the_same_bits(dtype, lens, heads):
    """Sequences that end while others go on: the CTAs behind them start beside warps in the midst of their chunks."""
    w = DeltaWorld(lens, heads=heads, heads_k=16, dtype=dtype, seed=15)
    state, batch = w.handles(D)
    n, want = len(lens), None
    for _ in range(12):
        o = torch.empty_like(w.v)
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
        got = (o.view(torch.int16), w.pool[n:2 * n].view(torch.int32).clone())
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert D.delta_device_error() == 0 and torch.isfinite(o).all()


@pytest.mark.parametrize("dim_k", [64, 128])
@pytest.mark.parametrize("lens", [[300], [300, 20, 9, 12, 40, 1, 0, 33], [20, 9, 300, 8, 150, 300, 1], [40] * 12, [9] * 126 + [70, 33],
                                  [9] * 127 + [70, 33]])
def test_shapes_of_a_batch(dim_k, lens):
    """One long sequence, a few among short ones, all alike, as many as are put in order and one more."""
    DeltaWorld(lens, heads=8, heads_k=4, dim_k=dim_k, seed=16).check(D)


@pytest.mark.parametrize("lens", [[300, 20, 9, 12], [40] * 30, [5, 300]])
def test_a_bound_far_above_the_lengths(lens):
    DeltaWorld(lens, heads=16, heads_k=8, seed=17).check(D, max_q=100_000)
