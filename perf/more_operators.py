"""More operators of the verifying model under measurement: attention of a batch whose sequences
share long beginnings, and the gated delta rule of recurrent layers, token by token and over
whole prompts.

``run`` computes an operator from elementary torch operations in 32 bits (sums of log decays in
64), or, with ``own`` set, through this repository's entry points.  Lengths are a function of the
case, values of the seed.
"""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
CHUNK = 64                     # of the plain form of the delta rule


def listed():
    heads = {"heads": 32, "kv_heads": 8, "dim": 128}
    delta = {"op": "delta", "heads": 32, "k_heads": 16, "dim_k": 128, "dim_v": 128, "fresh": 0, "branches": 0, "save": 0}
    return [
        # four continuations of a short prompt, a token each: the smallest call, where latency counts
        {"name": "shared_decode_small", "op": "shared", "n_prefix": 1, "prefix": 1024, "n_seq": 4, "q": 1, "ragged": 0,
         "own_lo": 1, "own_hi": 64, "page": 16, "format": "f16", "dtype": "f16", "mask": "causal", **heads},
        # 64 samples drawn from one long prompt, a token each
        {"name": "shared_decode_64", "op": "shared", "n_prefix": 1, "prefix": 16384, "n_seq": 64, "q": 1, "ragged": 0,
         "own_lo": 1, "own_hi": 1024, "page": 16, "format": "bf16", "dtype": "bf16", "mask": "causal", **heads},
        # drafted blocks of 48 requests behind three system prompts of uneven length, 64-wide heads
        {"name": "shared_verify_groups", "op": "shared", "n_prefix": 3, "prefix": 8191, "n_seq": 48, "q": 9, "ragged": 1,
         "own_lo": 9, "own_hi": 2048, "page": 32, "format": "f16", "dtype": "f16", "mask": "causal",
         "heads": 32, "kv_heads": 8, "dim": 64},
        # token trees of 16 samples over an int8 cache
        {"name": "shared_tree_int8", "op": "shared", "n_prefix": 1, "prefix": 8192, "n_seq": 16, "q": 31, "ragged": 1,
         "own_lo": 31, "own_hi": 512, "page": 32, "format": "int8", "dtype": "bf16", "mask": "tree", **heads},
        # eight questions of 256 tokens about one long document
        {"name": "shared_questions_long", "op": "shared", "n_prefix": 1, "prefix": 32768, "n_seq": 8, "q": 256,
         "ragged": 0, "own_lo": 256, "own_hi": 256, "page": 64, "format": "bf16", "dtype": "bf16", "mask": "causal",
         **heads},
        # one sequence, one token
        {"name": "delta_step_one", **delta, "n_seq": 1, "q": 1, "ragged": 0, "dtype": "bf16"},
        # a token each of 64 sequences
        {"name": "delta_step_64", **delta, "n_seq": 64, "q": 1, "ragged": 0, "dtype": "bf16"},
        # drafted blocks of 64 samples that branch from one prompt's state, the state kept after every token
        {"name": "delta_verify_save", **delta, "n_seq": 64, "q": 9, "ragged": 1, "dtype": "f16", "branches": 1, "save": 1},
        # blocks verified without keeping states between
        {"name": "delta_verify_32", **delta, "n_seq": 32, "q": 16, "ragged": 1, "dtype": "bf16"},
        # prompt chunks among single tokens, heads of 64
        {"name": "delta_mixed_64", **delta, "n_seq": 16, "q": 1000, "ragged": 2, "dtype": "f16", "dim_k": 64, "dim_v": 64},
        # one long prompt from its first token
        {"name": "delta_prompt_one", **delta, "n_seq": 1, "q": 16381, "ragged": 0, "dtype": "bf16", "fresh": 1},
        # a batch of prompts that go on from a state
        {"name": "delta_prompts", **delta, "n_seq": 8, "q": 4096, "ragged": 1, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.5:
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
        h, hk = rng.choice([(32, 16), (32, 32), (16, 16), (48, 16), (8, 4)])
        n = _log_int(rng, 1, 64)
        q = _log_int(rng, 1, max(1, min(16384, 32768 * 32 // (n * h))))
        return {"op": "delta", "heads": h, "k_heads": hk, "dim_k": dk, "dim_v": dv, "n_seq": n, "q": q,
                "ragged": rng.choice([0, 1, 2]), "dtype": rng.choice(["f16", "bf16"]), "fresh": rng.choice([0, 0, 1]),
                "branches": rng.choice([0, 0, 1]), "save": rng.choice([0, 1]) if q <= 16 else 0}
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 16), (28, 4), (40, 8)])
    dtype = rng.choice(["f16", "bf16"])
    mask = rng.choice(["causal", "causal", "full", "tree"])
    q = _log_int(rng, 1, 40 if mask == "tree" else 256)
    n = _log_int(rng, 2, max(2, min(64, 1024 // q)))
    prefix = _log_int(rng, 16, 32768)
    return {"op": "shared", "n_prefix": rng.choice([1, 1, 2, min(5, n)]), "prefix": prefix, "n_seq": n, "q": q,
            "ragged": rng.choice([0, 1, 2]), "own_lo": q, "own_hi": q + _log_int(rng, 1, 2048),
            "page": rng.choice([16, 32, 64, 128]), "format": rng.choice([dtype, "int8", "e4m3"]), "dtype": dtype,
            "mask": mask, "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128])}


# ---------------------------------------------------------------------------- lengths

def _spread(n, lo, hi, turn):
    """n whole numbers over [lo, hi], the largest first, the others by the golden ratio."""
    return [hi if i == 0 else lo + int((i * 0.6180339887498949 + turn) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _new(case):
    """New tokens of each sequence."""
    n, q = case["n_seq"], case["q"]
    if case["ragged"] == 0:
        return [q] * n
    if case["ragged"] == 1:                      # anything up to q
        return _spread(n, 1, q, 0.35)
    return [max(1, q - 37 * i) if i % 4 == 0 else 1 for i in range(n)]     # one chunk in four, single tokens besides


def _starts(new):
    return [sum(new[:i]) for i in range(len(new) + 1)]


def _shared_lengths(case):
    """New tokens and own cached tokens (with the new ones) of each sequence; of each prefix its length and the first
    sequence that has it."""
    new = _new(case)
    kv = _spread(case["n_seq"], case["own_lo"], case["own_hi"], 0.0)
    p = case["n_prefix"]
    return ([min(a, b) for a, b in zip(new, kv)], kv, _spread(p, max(1, case["prefix"] // 3), case["prefix"], 0.2),
            [i * case["n_seq"] // p for i in range(p + 1)])


# ---------------------------------------------------------------------------- inputs

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(gen, n_pages, case):
    """One pool [n_pages, kv_heads, page, dim] in the case's format and its row scales."""
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=gen)
    if case["format"] in DTYPES:
        return x.to(DTYPES[case["format"]]), None
    if case["format"] == "int8":
        codes, unit = (x * 36).clamp_(-127, 127).round_().to(torch.int8), 36
    else:
        codes, unit = (x * 128).clamp_(-448, 448).to(torch.float8_e4m3fn), 128
    return codes, (torch.rand(shape[:3], device="cuda", generator=gen) * 0.4 + 0.8) / unit


def _table(lengths, page, ids):
    """Block table of sequences of some lengths from a run of page numbers."""
    used = [-(-x // page) for x in lengths]
    pages = torch.full((len(used), max(used)), -1, dtype=torch.int32, device="cuda")
    pages[torch.arange(max(used), device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]] = ids
    return pages


def _prepare_shared(case, gen):
    new, kv, long, first = _shared_lengths(case)
    page, t, dt = case["page"], sum(new), DTYPES[case["dtype"]]
    a, b = (sum(-(-x // page) for x in y) for y in (kv, long))
    ids = torch.randperm(a + b, device="cuda", generator=gen).to(torch.int32)
    start = _starts(new)
    s = {"case": case, "q_start": _ints(start), "kv_len": _ints(kv), "pages": _table(kv, page, ids[:a]),
         "p_start": _ints([start[i] for i in first]), "p_len": _ints(long), "p_pages": _table(long, page, ids[a:]),
         "max_q": max(new), "max_kv": max(kv), "p_max_q": max(start[j] - start[i] for i, j in zip(first, first[1:])),
         "p_max_kv": max(long)}
    s["k_pool"], s["k_scale"] = _pool(gen, a + b, case)
    s["v_pool"], s["v_scale"] = _pool(gen, a + b, case)
    s["q"] = torch.randn(t, case["heads"], case["dim"], device="cuda", dtype=dt, generator=gen)
    s["o"] = torch.empty_like(s["q"])
    if case["mask"] == "tree":
        # node j sees itself and a random part of the nodes before it
        i = torch.arange(t, device="cuda") - s["q_start"][_owner(s["q_start"], t)]
        bits = torch.randint(0, 1 << 62, (t,), device="cuda", generator=gen)
        one = torch.ones_like(bits)
        s["tree"] = (bits & ((one << i) - 1)) | (one << i)
    if own:  # the handles over the cache and the batch that a serving program keeps
        from speculative_decoding_draft_kv_gb300 import paged
        s["cache"] = paged.PagedCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        s["batch"] = paged.PagedBatch(s["q_start"], s["kv_len"], s["pages"], s["max_q"], s["max_kv"])
        s["prefix"] = paged.PagedBatch(s["p_start"], s["p_len"], s["p_pages"], s["p_max_q"], s["p_max_kv"])
        n = paged.paged_attend_shared_workspace(s["cache"], s["batch"], s["prefix"], t, case["heads"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


def _prepare_delta(case, gen):
    new, n, dt = _new(case), case["n_seq"], DTYPES[case["dtype"]]
    t, h, hk, dk, dv = sum(new), case["heads"], case["k_heads"], case["dim_k"], case["dim_v"]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=gen)

    s = {"case": case, "q_start": _ints(_starts(new)), "max_q": max(new)}
    # one projection's queries, keys and values side by side
    wide = randn(t, 2 * hk * dk + h * dv, dtype=dt)
    s["q"] = wide[:, :hk * dk].view(t, hk, dk)
    s["k"] = wide[:, hk * dk:2 * hk * dk].view(t, hk, dk)
    s["v"] = wide[:, 2 * hk * dk:].view(t, h, dv)
    # decays mostly near 1, heads of several time scales; weights of the update between 0 and 1
    rate = torch.exp(randn(h) - 2.5)
    s["g"] = -rate * torch.nn.functional.softplus(randn(t, h))
    s["beta"] = torch.sigmoid(randn(t, h))
    s["o"] = torch.empty(t, h, dv, device="cuda", dtype=dt)
    # the states' pool: those that are read, then those that are written
    read = 0 if case["fresh"] else (1 if case["branches"] else n)
    write = t if case["save"] else n
    s["state"] = randn(read + write, h, dv, dk) * 0.2
    order = torch.randperm(read + write, device="cuda", generator=gen).to(torch.int32)
    none = torch.full((n,), -1, device="cuda", dtype=torch.int32)
    s["slot_in"] = none if case["fresh"] else (order[:1].expand(n).contiguous() if case["branches"] else order[:n].contiguous())
    s["slot_out"] = none if case["save"] else order[read:].contiguous()
    s["save"] = order[read:].contiguous() if case["save"] else None
    if own:  # handles over the states and the batch, and a workspace
        from speculative_decoding_draft_kv_gb300 import delta
        s["states"] = delta.DeltaState(s["state"])
        s["batch"] = delta.DeltaBatch(s["q_start"], s["slot_in"], s["slot_out"], s["max_q"], save=s["save"])
        n = delta.delta_rule_workspace(s["states"], s["batch"], t, hk)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_shared(case, gen) if case["op"] == "shared" else _prepare_delta(case, gen)


# ---------------------------------------------------------------------------- plain forms

def _owner(start, t):
    """The sequence of each row."""
    return torch.searchsorted(start[1:].contiguous(), torch.arange(t, device="cuda", dtype=torch.int32), right=True)


def _keys(s, pages, length, name):
    """K or V of some block table [n, kv_heads, max length, dim] in 32 bits, zeros behind each length."""
    page = s["case"]["page"]
    p = torch.arange(int(pages.shape[1]) * page, device="cuda")
    ids = pages[:, p // page].clamp(min=0).long()
    slot = (p % page)[None].expand_as(ids)
    pool, scale = s[name + "_pool"], s[name + "_scale"]
    if scale is None:
        x = pool[ids, :, slot].float()
    else:
        x = pool.view(torch.uint8)[ids, :, slot].view(pool.dtype).float() * scale[ids, :, slot][..., None]
    return torch.where((p[None] < length[:, None])[..., None, None], x, 0.0).permute(0, 2, 1, 3)


def _part(s, start, most, pages, length, see):
    """Softmax state of all rows over one block table: (largest score, sum, numerators) by row and head.
    see(i, p): truth values [n, most, positions]."""
    c = s["case"]
    group, d, g = c["heads"] // c["kv_heads"], c["dim"], c["kv_heads"]
    k, v = _keys(s, pages, length, "k"), _keys(s, pages, length, "v")
    n, lk, t = k.shape[0], k.shape[2], s["q"].shape[0]
    i = torch.arange(most, device="cuda")
    row = (start[:-1, None] + i).clamp(max=t - 1).long()
    q = s["q"][row].float().view(n, most, g, group, d).permute(0, 2, 3, 1, 4).reshape(n, g, group * most, d)
    visible = see(i[None, :, None], torch.arange(lk, device="cuda")[None, None])[:, None, None]
    score = (q @ k.transpose(2, 3)).view(n, g, group, most, lk).mul_(d ** -0.5)
    score.masked_fill_(~visible, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1)
    acc = (score.view(n, g, group * most, lk) @ v).view(n, g, group, most, d)
    r = torch.arange(t, device="cuda")
    at = _owner(start, t)
    place = r - start[at]
    flat = [x.permute(0, 3, 1, 2, *range(4, x.dim()))[at, place].reshape(t, c["heads"], *x.shape[4:])
            for x in (top[..., 0], total, acc)]
    return flat


def _plain_shared(s):
    c = s["case"]
    new = (s["q_start"][1:] - s["q_start"][:-1])[:, None, None]
    kv = s["kv_len"][:, None, None]
    context = kv - new

    def see_own(i, p):
        if c["mask"] == "causal":
            see = p <= context + i
        elif c["mask"] == "full":
            see = p < kv
        else:
            word = s["tree"][(s["q_start"][:-1, None, None] + i).clamp(max=s["tree"].numel() - 1).long()]
            see = (p < context) | ((p < kv) & ((word >> (p - context).clamp(0, 62)) & 1).bool())
        return see & (i < new)

    m0, l0, a0 = _part(s, s["p_start"], s["p_max_q"], s["p_pages"], s["p_len"],
                       lambda i, p: (p < s["p_len"][:, None, None]).expand(-1, s["p_max_q"], -1))
    m1, l1, a1 = _part(s, s["q_start"], s["max_q"], s["pages"], s["kv_len"], see_own)
    m = torch.maximum(m0, m1)
    w0, w1 = torch.exp(m0 - m), torch.exp(m1 - m)
    s["o"].copy_((a0 * w0[..., None] + a1 * w1[..., None]) / (l0 * w0 + l1 * w1)[..., None])
    return {"o": s["o"]}


def _inverse(low):
    """(I + low)^-1 of strictly lower triangular matrices [..., C, C], C a power of two: inverses of the diagonal's
    blocks, two neighbours of each size put together."""
    c = low.shape[-1]
    inv = torch.eye(c, device=low.device, dtype=low.dtype).expand_as(low).clone()
    size = 1
    while size < c:
        n = c // (2 * size)
        blocks = low.unflatten(-1, (n, 2, size)).unflatten(-4, (n, 2, size))           # [..., n, 2, size, n, 2, size]
        e = torch.arange(n, device=low.device)
        view = inv.unflatten(-1, (n, 2, size)).unflatten(-4, (n, 2, size))
        a, b = view[..., e, 0, :, e, 0, :], view[..., e, 1, :, e, 1, :]
        view[..., e, 1, :, e, 0, :] = -(b @ blocks[..., e, 1, :, e, 0, :] @ a)
        size *= 2
    return inv


def _plain_delta(s):
    c = s["case"]
    start, t, most = s["q_start"], s["q"].shape[0], s["max_q"]
    n, h, dk, dv = c["n_seq"], c["heads"], c["dim_k"], c["dim_v"]
    size = min(CHUNK, 1 << max(0, most - 1).bit_length())
    chunks = -(-most // size)
    i = torch.arange(chunks * size, device="cuda")
    row = (start[:-1, None] + i).clamp(max=t - 1).long()
    alive = (i[None] < (start[1:] - start[:-1])[:, None])

    def padded(x):
        """[t, heads, ...] -> [chunks, n, h, size, ...], zeros behind each sequence."""
        x = torch.where(alive.view(*alive.shape, *[1] * (x.dim() - 1)), x[row], 0.0)
        x = x.repeat_interleave(h // x.shape[2], 2).unflatten(1, (chunks, size))
        return x.permute(1, 0, 3, 2, *range(4, x.dim()))

    def unit(x):
        x = x.float()
        return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)

    q, k, v = padded(unit(s["q"])) * dk ** -0.5, padded(unit(s["k"])), padded(s["v"].float())
    beta, total = padded(s["beta"])[..., None], padded(s["g"]).double().cumsum(-1)
    lower = torch.ones(size, size, device="cuda", dtype=torch.bool).tril()
    decay = torch.where(lower, total[..., :, None] - total[..., None, :], -math.inf).exp().float()
    gone = total.exp().float()[..., None]                                      # since the chunk's beginning
    left = (total[..., -1:] - total).exp().float()[..., None]                  # until its end
    inv = _inverse((k @ k.transpose(-1, -2) * decay * beta).tril(-1))
    inner = q @ k.transpose(-1, -2) * decay
    state = torch.zeros(n, h, dk, dv, device="cuda")
    if not c["fresh"]:
        state = s["state"][s["slot_in"].long()].transpose(-1, -2)
    out = torch.empty_like(v)
    for j in range(chunks):
        u = inv[j] @ (beta[j] * (v[j] - gone[j] * (k[j] @ state)))
        out[j] = gone[j] * (q[j] @ state) + inner[j] @ u
        before = state
        state = state * gone[j][..., -1:, :] + (k[j] * left[j]).transpose(-1, -2) @ u
    owner = _owner(start, t)
    place = torch.arange(t, device="cuda") - start[owner]
    s["o"].copy_(out.permute(1, 0, 3, 2, 4).flatten(1, 2)[owner, place])
    if c["save"]:                                                              # one chunk: after each of its tokens
        weights = (decay[0][..., None] * k[0][..., None, :, :]).transpose(-1, -2)   # [n, h, token, dk, size]
        every = before[:, :, None] * gone[0][..., None] + weights @ u[:, :, None]
        s["state"][s["save"].long()] = every.transpose(-1, -2).transpose(1, 2)[owner, place]
    else:
        s["state"][s["slot_out"].long()] = state.transpose(-1, -2)
    return {"o": s["o"], "state": s["state"]}


def run(state):
    if own:
        return _own(state)
    return _plain_shared(state) if state["case"]["op"] == "shared" else _plain_delta(state)


def _own(s):
    c = s["case"]
    if c["op"] == "shared":
        from speculative_decoding_draft_kv_gb300 import paged
        paged.paged_attend_shared(s["cache"], s["batch"], s["prefix"], s["q"], s["o"], mask=c["mask"],
                                  tree=s.get("tree"), workspace=s["workspace"])
        return {"o": s["o"]}
    from speculative_decoding_draft_kv_gb300 import delta
    delta.delta_rule(s["states"], s["batch"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], normalise=True, eps=EPS,
                     workspace=s["workspace"])
    return {"o": s["o"], "state": s["state"]}


# ---------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "delta":
        new, h, dk, dv = _new(case), case["heads"], case["dim_k"], case["dim_v"]
        t, n = sum(new), case["n_seq"]
        read = 0 if case["fresh"] else (1 if case["branches"] else n)
        rows = t * (2 * 2 * case["k_heads"] * dk + 2 * 2 * h * dv + 8 * h)
        return {"bytes": rows + 4 * h * dk * dv * (read + (t if case["save"] else n)), "flops": 6 * t * h * dk * dv}
    d, h, g = case["dim"], case["heads"], case["kv_heads"]
    row = 2 * g * (2 * d if case["format"] in DTYPES else d + 4)         # K and V of one token in the cache
    new, kv, long, first = _shared_lengths(case)
    pairs = sum(sum(new[a:b]) * p for a, b, p in zip(first, first[1:], long))
    for n, l in zip(new, kv):
        inner = {"causal": n * (n + 1) // 2, "full": n * n, "tree": n * (n + 3) // 4}[case["mask"]]
        pairs += n * (l - n) + inner
    return {"bytes": row * (sum(kv) + sum(long)) + 2 * 2 * sum(new) * h * d, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------- 64 bits

def _exact_rows(s, name, ids, length):
    """One block table's cached rows [length, kv_heads, dim], page after page."""
    ids = ids.long().clamp(min=0)
    pool, scale = s[name + "_pool"], s[name + "_scale"]
    if scale is None:
        x = pool[ids].double()
    else:
        x = pool.view(torch.uint8)[ids].view(pool.dtype).double() * scale[ids].double()[..., None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:length]


def _exact_shared(case, s):
    new, kv, long, first = _shared_lengths(case)
    start, group = _starts(new), case["heads"] // case["kv_heads"]
    out = torch.empty(sum(new), case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    for p, length in enumerate(long):
        shared = [_exact_rows(s, a, s["p_pages"][p], length) for a in "kv"]
        for i in range(first[p], first[p + 1]):
            k, v = (torch.cat([x, _exact_rows(s, a, s["pages"][i], kv[i])]) for x, a in zip(shared, "kv"))
            n, c = new[i], kv[i] - new[i]
            tok, pos = torch.arange(n, device="cuda")[:, None], torch.arange(kv[i], device="cuda")
            hidden = torch.zeros(n, kv[i], dtype=torch.bool, device="cuda")
            if case["mask"] == "causal":
                hidden = pos > c + tok
            elif case["mask"] == "tree":
                word = s["tree"][start[i]:start[i + 1], None]
                hidden[:, c:] = ((word >> torch.arange(n, device="cuda")) & 1) == 0
            hidden = torch.cat([torch.zeros(n, length, dtype=torch.bool, device="cuda"), hidden], 1)
            q = s["q"][start[i]:start[i + 1]].double()
            for j in range(case["heads"]):
                z = (q[:, j] @ k[:, j // group].T) / math.sqrt(case["dim"])
                out[start[i]:start[i + 1], j] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[:, j // group]
    return {"o": out}


def _exact_delta(case, s):
    """Token by token, the sequences that still have one side by side."""
    new, h, dk = _new(case), case["heads"], case["dim_k"]
    start = torch.tensor(_starts(new), device="cuda")
    pool = s["state"].double()
    out = torch.empty(s["o"].shape, dtype=torch.float64, device="cuda")
    if case["fresh"]:
        state = torch.zeros(case["n_seq"], *pool.shape[1:], dtype=torch.float64, device="cuda")
    else:
        state = pool[s["slot_in"].long()]                                      # [n, h, dv, dk]
    counts = torch.tensor(new)
    for j in range(max(new)):
        who = (counts > j).nonzero()[:, 0].cuda() if case["ragged"] else None
        r = start[:-1] + j if who is None else start[who] + j
        x = state if who is None else state[who]
        q, k = (a[r].double().repeat_interleave(h // case["k_heads"], 1) for a in (s["q"], s["k"]))
        q, k = (a / (a.square().sum(-1, keepdim=True) + EPS).sqrt() for a in (q, k))
        x = x * torch.exp(s["g"][r].double())[..., None, None]
        u = s["beta"][r].double()[..., None] * (s["v"][r].double() - (x @ k[..., None])[..., 0])
        x = x + u[..., :, None] * k[..., None, :]
        out[r] = (x @ q[..., None])[..., 0] / math.sqrt(dk)
        if case["save"]:
            pool[s["save"][r].long()] = x
        if who is None:
            state = x
        else:
            state[who] = x
    if not case["save"]:
        pool[s["slot_out"].long()] = state
    return {"o": out, "state": pool}


def exact(case, seed):
    if case["op"] == "shared" and work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    return _exact_shared(case, s) if case["op"] == "shared" else _exact_delta(case, s)
