"""delta_rule against its float64 form: types, sizes, head groups, lengths around the kernels' blocks, states
that are read by several, written in place or kept behind every token, and what must not matter."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import delta as D
from tests.delta_oracle import DeltaWorld

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dims", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [[1], [8], [1, 0, 9], [7, 16, 2], [33, 1, 64], [130]])
def test_types_sizes_and_lengths(dtype, dims, lens):
    DeltaWorld(lens, dim_k=dims[0], dim_v=dims[1], dtype=dtype, spare_rows=2, seed=sum(lens)).check(D)


@pytest.mark.parametrize("heads,heads_k", [(1, 1), (4, 4), (3, 1), (32, 16), (6, 2)])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_head_groups(heads, heads_k, n):
    DeltaWorld([n, n + 1], heads=heads, heads_k=heads_k, seed=heads + n).check(D)


@pytest.mark.parametrize("n", list(range(1, 20)) + [31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200])
def test_every_small_length(n):
    DeltaWorld([n], heads=2, heads_k=1, dtype=F16, seed=n).check(D)


@pytest.mark.parametrize("n", [3, 50])
def test_without_a_state(n):
    w = DeltaWorld([n, n], seed=1)
    w.slot_in = [-1, -5]
    w.pool[:2] = math.nan
    w.check(D)


@pytest.mark.parametrize("n", [2, 70])
def test_branches_read_one_slot(n):
    w = DeltaWorld([n, n - 1, 1, 0, n], seed=2)
    w.slot_in = [1] * 5
    w.check(D)


@pytest.mark.parametrize("n", [1, 9, 80])
def test_in_place_and_not_kept(n):
    w = DeltaWorld([n, n, n], seed=3)
    w.slot_out = [0, -1, 2]
    w.check(D)


@pytest.mark.parametrize("lens", [[9, 4, 0, 1], [40, 3]])
@pytest.mark.parametrize("final", [True, False])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_states_behind_every_token(lens, final, dtype):
    n = len(lens)
    w = DeltaWorld(lens, dtype=dtype, slots=2 * n + sum(lens) + 1, seed=4, spare_rows=1)
    w.save = [2 * n + r for r in range(w.total)] + [0]        # the spare row's is not looked at
    if not final:
        w.slot_out = [-1] * n
    w.check(D)
    w.save = [x if i % 3 else -1 for i, x in enumerate(w.save)]
    w.check(D)


def test_rollback_goes_on_from_the_last_accepted_token():
    """A block whose tail is rejected: the next block begins from the state behind the accepted part, and
    what comes out is what the accepted tokens alone give."""
    n, take = 8, 5
    w = DeltaWorld([n], slots=n + 3, seed=5)
    w.save, w.slot_out = [3 + i if i < n else -1 for i in range(n)], [-1]
    w.check(D)
    x = DeltaWorld([take + 4], seed=6)
    for a in ("q", "k", "v", "decay", "beta"):
        getattr(x, a)[:take] = getattr(w, a)[:take]
    x.pool[0] = w.pool[0]
    o = x.check(D)
    y = DeltaWorld([4], seed=7, slots=n + 3)
    for a in ("q", "k", "v", "decay", "beta"):
        setattr(y, a, getattr(x, a)[take:].contiguous())
    y.pool = w.pool
    y.slot_in, y.slot_out = [3 + take - 1], [1]
    oy = y.check(D)
    assert (o[take:].double() - oy.double()).abs().max() <= 2 ** -7 * o.double().abs().max()


@pytest.mark.parametrize("lens", [[1, 3], [100]])
def test_strides(lens):
    """Slices of one projection, heads inside wider rows, a pool of another order."""
    w = DeltaWorld(lens, heads=4, heads_k=2, seed=8)
    t = w.rows
    wide = torch.full((t, 2 * 128 * 2 + 4 * 128 + 64), math.nan, dtype=w.dtype, device="cuda")
    for name, at, heads in (("q", 0, 2), ("k", 256, 2), ("v", 512, 4)):
        part = wide[:, at:at + heads * 128].view(t, heads, 128)
        part.copy_(getattr(w, name))
        setattr(w, name, part)
    both = torch.full((t, 11), math.nan, device="cuda")
    for name, at in (("decay", 1), ("beta", 6)):
        part = both[:, at:at + 4]
        part.copy_(getattr(w, name))
        setattr(w, name, part)
    pool = torch.full((4, w.n_slots + 1, 128, 128), math.nan, device="cuda").transpose(0, 1)[1:]
    pool.copy_(w.pool)
    w.pool = pool
    o = torch.full((t, 6, 136), 7.0, dtype=w.dtype, device="cuda")
    w.check(D, o=o[:, 1:5, :128])
    assert (o[:, 0] == 7).all() and (o[:, 5] == 7).all() and (o[:, :, 128:] == 7).all()


@pytest.mark.parametrize("n", [6, 75])
def test_keys_as_they_are(n):
    """Without norms: unit keys come from the caller, queries of any length."""
    w = DeltaWorld([n, n], seed=9)
    w.k = torch.nn.functional.normalize(w.k.float(), dim=-1).to(w.dtype)
    w.check(D, normalise=False, scale=0.37)


@pytest.mark.parametrize("n", [5, 90])
def test_eps_counts_for_short_keys(n):
    w = DeltaWorld([n], seed=10)
    w.k[::2] *= 1e-3
    w.check(D, eps=1e-2)
    w.k[1] = 0
    w.q[2] = 0
    w.check(D, eps=0.0625)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [7, 100])
def test_the_same_key_again_and_again(dtype, n):
    """Every key alike and beta up to 1 and 2: the update's system is as far from diagonal as it gets."""
    for top in (1.0, 2.0):
        w = DeltaWorld([n], dtype=dtype, seed=11, rate=1e-3)
        w.k[:n] = w.k[:1].clone()
        w.beta[:n] = top
        w.check(D)


@pytest.mark.parametrize("n", [12, 140])
def test_decays_from_none_to_all(n):
    """No decay, tiny and huge ones, and a state that is dropped in the middle: what follows keeps its precision."""
    w = DeltaWorld([n], heads=6, heads_k=2, seed=12)
    w.decay[:n, 0] = 0.0
    w.decay[:n, 1] = -1e-6
    w.decay[:n, 2] = -30.0
    w.decay[n // 2, 3] = -math.inf
    w.decay[n // 3, 4] = -3.4e38
    w.decay[n // 3:n // 2 + 2, 5] = -1e4
    w.check(D)


@pytest.mark.parametrize("n", [3, 66])
@pytest.mark.parametrize("spread", [1e-6, 3e3, 1e12])
def test_far_magnitudes(n, spread):
    """States and values far below and above 1 (bf16 has the range), head by head."""
    w = DeltaWorld([n], dtype=BF16, spread=spread, seed=13)
    w.v[:n, 1] *= 2.0 ** -20
    w.pool[0, 2] *= 2.0 ** -20
    w.check(D)


@pytest.mark.parametrize("n", [4, 70])
def test_bf16_keys_of_any_magnitude(n):
    w = DeltaWorld([n], dtype=BF16, seed=14)
    w.k *= 2.0 ** (torch.arange(w.rows, device="cuda") % 40 - 20)[:, None, None]
    w.q *= 2.0 ** 30
    w.check(D, eps=0.0)


@pytest.mark.parametrize("n", [3, 100])
def test_nan_and_infinities_stay_in_their_heads_and_sequences(n):
    w = DeltaWorld([n, n], heads=4, heads_k=4, seed=15)
    out, tol, slots = w.want()
    w.v[1, 0, 5] = math.nan
    w.k[n + 1, 2, 3] = math.inf
    w.pool[0, 3, 7, 7] = math.inf
    state, batch = w.handles(D)
    o = torch.empty(w.rows, 4, w.dim_v, dtype=w.dtype, device="cuda")
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
    assert D.delta_device_error() == 0
    off = (o.double() - out).abs() <= tol
    for s in range(2):
        r = slice(s * n, s * n + n)
        for h in range(4):
            clean = (s, h) not in ((0, 0), (1, 2), (0, 3))
            if clean:
                assert off[r, h].all()
                S, bound = slots[2 + s]
                assert torch.linalg.matrix_norm(w.pool[2 + s, h].double() - S[h]) <= bound[h]
    assert torch.isnan(w.pool[2, 0, 5]).all()             # the value element that was NaN
    assert not torch.isfinite(w.pool[3, 2]).any()         # a key with an infinity has no norm
    if n == 3:                                            # (long runs: see the header)
        assert off[0, 0].all() and off[n, 2].all()        # tokens in front of it


def test_empty_batches_and_sequences():
    w = DeltaWorld([0, 0], seed=16)
    w.check(D)                                             # states are copied
    w = DeltaWorld([0, 3, 0], spare_rows=4, seed=17)
    w.check(D, max_q=11)
    w = DeltaWorld([2], seed=18)
    state, _ = w.handles(D)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    batch = D.DeltaBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), none, none, 4)
    o = torch.full_like(w.v, 7.0)
    D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
    assert D.delta_device_error() == 0 and (o == 7).all()


@pytest.mark.parametrize("n", [2, 50])
def test_broken_batches_are_left_alone(n):
    lens = [n] * 4

    def run(q_start=None, max_q=None, slot_in=None, slot_out=None, save=None):
        w = DeltaWorld(lens, slots=20, seed=19)
        w.slot_in = slot_in or w.slot_in
        w.slot_out = slot_out or w.slot_out
        w.save = save
        state, batch = w.handles(D, max_q)
        if q_start is not None:
            batch = D.DeltaBatch(w.ints(q_start), batch.tensors[1], batch.tensors[2], max_q or n)
        before, o = w.pool.clone(), torch.full_like(w.v, 7.0)
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
        bits = D.delta_device_error()
        same = [torch.equal(w.pool[i].view(torch.int32), before[i].view(torch.int32)) for i in range(20)]
        return w, o, bits, same

    for q_start, alone in (([0, n, n - 1, n, 2 * n], 1), ([0, n, 2 * n, 3 * n, 4 * n + 1], 3), ([-1, n, 2 * n, 3 * n, 4 * n], 0),
                           ([0, n - 1, 2 * n, 3 * n, 4 * n], 1)):
        w, o, bits, same = run(q_start)
        assert bits == D.DELTA_ERR_BATCH
        assert same[4 + alone] and not same[4 + (alone + 2) % 4]
    w, o, bits, same = run(slot_in=[0, 20, 2, 1 << 30])
    assert bits == D.DELTA_ERR_SLOT and same[5] and same[7] and not same[4]
    assert (o[n:2 * n] == 7).all() and (o[3 * n:] == 7).all() and (o[:n] != 7).any()
    w, o, bits, same = run(slot_out=[4, 20, 6, 1 << 30])
    assert bits == D.DELTA_ERR_SLOT and not same[4] and all(same[8:]) and (o[n:2 * n] != 7).any()
    w, o, bits, same = run(save=[25] * n + [9] * n + [-1] * (2 * n))
    assert bits == D.DELTA_ERR_SLOT and not same[9]


@pytest.mark.parametrize("n", [1, 6, 90])
def test_captured_and_replayed(n):
    """A replay follows the arrays: other lengths, slots and values."""
    w = DeltaWorld([n, n, n], seed=20, slots=12)
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
    for lens, slot_in, slot_out in (([n, n, n], [0, 1, 2], [3, 4, 5]), ([max(0, n - 1), n, 1], [2, -1, 2], [6, 7, -1])):
        x = DeltaWorld(lens, seed=21 + lens[0], slots=12, spare_rows=3 * n - sum(lens))
        for a in ("q", "k", "v", "decay", "beta"):
            getattr(w, a).copy_(getattr(x, a))
        w.pool.copy_(kept)
        x.pool.copy_(kept)
        x.slot_in, x.slot_out = slot_in, slot_out
        for to, src in zip(arrays, (x.q_start, x.ints(slot_in), x.ints(slot_out))):
            to.copy_(src)
        out, tol, slots = x.want()
        o.fill_(7.0)
        graph.replay()
        assert D.delta_device_error() == 0
        assert ((o[:x.total].double() - out).abs() <= tol).all() and (o[x.total:] == 7).all()
        for slot, (S, bound) in slots.items():
            assert (torch.linalg.matrix_norm(w.pool[slot].double() - S) <= bound).all()


def test_two_streams_at_once():
    worlds = [DeltaWorld([300, 5], seed=30), DeltaWorld([2, 3], seed=31)]
    streams = [torch.cuda.Stream() for _ in worlds]
    torch.cuda.synchronize()
    outs, wants = [], [w.want() for w in worlds]
    for w, st in zip(worlds, streams):
        state, batch = w.handles(D)
        torch.cuda.synchronize()
        o = torch.empty_like(w.v)
        torch.cuda.synchronize()
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o, stream=st)
        outs.append((o, state, batch))
    assert D.delta_device_error() == 0
    for w, (o, *_), (out, tol, slots) in zip(worlds, outs, wants):
        assert ((o.double() - out).abs() <= tol).all()
        for slot, (S, bound) in slots.items():
            assert (torch.linalg.matrix_norm(w.pool[slot].double() - S) <= bound).all()


@pytest.mark.parametrize("n", [5, 150])
def test_the_same_call_gives_the_same_bits(n):
    w = DeltaWorld([n, 2 * n], seed=32)
    state, batch = w.handles(D)
    got = []
    for _ in range(3):
        o = torch.empty_like(w.v)
        D.delta_rule(state, batch, w.q, w.k, w.v, w.decay, w.beta, o)
        got.append((o.view(torch.int16).clone(), w.pool[2:4].view(torch.int32).clone()))
    assert all(torch.equal(a, b) for x in got[1:] for a, b in zip(x, got[0]))


def test_many_sequences():
    """More CTAs than fit at once, and a pool whose offsets pass 32 bits."""
    n, heads = 700, 32
    w = DeltaWorld([1] * n, heads=heads, heads_k=8, seed=33, slots=n + 1400)   # 2,100 slots of 2 MB
    w.slot_out = list(range(2 * n - 1, n - 1, -1))
    w.slot_out[0] = n + 1399
    w.check(D)


@pytest.mark.parametrize("n", [1, 5, 40])
def test_a_pool_past_32_bits(n):
    """Slots 2^30 floats apart: the last one's byte offset is past 2^33, its element offset past 2^31."""
    w = DeltaWorld([n, n], slots=4, seed=21)
    far = torch.empty(3 * (1 << 30) + w.pool[0].numel(), device="cuda")
    pool = far.as_strided(w.pool.shape, (1 << 30, *w.pool.stride()[1:]))
    pool.copy_(w.pool)
    w.pool = pool
    w.slot_in, w.slot_out = [0, 1], [2, 3]
    w.check(D)
