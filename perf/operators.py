"""The paged-cache operators under measurement: head norms with the position rotation, writing
and reading a quantised cache, and attention of new tokens over its pages.

``run`` computes an operator from elementary torch operations in 32 bits (angles in 64), or,
with ``own`` set, through this repository's entry points.  Lengths are a function of the case,
values of the seed.
"""

import math

import torch

own = False

EPS = 1e-6
THETA = 1.0e6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


def listed():
    heads = {"heads": 32, "kv_heads": 8, "dim": 128}
    return [
        # the verify block of one sequence (8 drafted tokens): norms and rotation on their own
        {"name": "norm_rope_verify_block", "op": "norm_rope", "rows": 8, "dtype": "f16", "rotary": 128,
         "layout": "half", "scaling": "none", **heads},
        # a prompt's projections, rotated over part of the head with frequencies scaled for long contexts
        {"name": "norm_rope_prompt", "op": "norm_rope", "rows": 16381, "dtype": "bf16", "rotary": 64,
         "layout": "interleaved", "scaling": "yarn", **heads},
        # one verification step of 64 sequences: queries and keys normed and rotated, K and V written as e4m3
        {"name": "append_step_e4m3", "op": "append", "n_seq": 64, "q": 9, "ragged": 1, "kv_lo": 9, "kv_hi": 256,
         "page": 16, "format": "e4m3", "dtype": "bf16", "fused": 1, "rotary": 128, "layout": "half",
         "scaling": "none", "read": 0, **heads},
        # a prompt's K and V quantised into int8 pages and read back (a cache moved to another holder)
        {"name": "append_read_int8", "op": "append", "n_seq": 4, "q": 8191, "ragged": 1, "kv_lo": 8191,
         "kv_hi": 12000, "page": 64, "format": "int8", "dtype": "f16", "fused": 0, "rotary": 128,
         "layout": "half", "scaling": "none", "read": 1, **heads},
        # one sequence's int8 cache read back
        {"name": "gather_one_int8", "op": "gather", "n_seq": 1, "kv_lo": 4096, "kv_hi": 4096, "page": 16,
         "format": "int8", "dtype": "f16", **heads},
        # every sequence of a batch read back from e4m3 pages
        {"name": "gather_batch_e4m3", "op": "gather", "n_seq": 64, "kv_lo": 1, "kv_hi": 8192, "page": 32,
         "format": "e4m3", "dtype": "bf16", **heads},
        # one sequence, one token: the smallest call of a serving loop
        {"name": "attend_decode_one", "op": "attend", "n_seq": 1, "q": 1, "ragged": 0, "kv_lo": 4096,
         "kv_hi": 4096, "page": 16, "format": "f16", "dtype": "f16", "mask": "causal", "window": 0, **heads},
        # verification of drafted blocks of 64 sequences of all lengths
        {"name": "attend_verify_64", "op": "attend", "n_seq": 64, "q": 9, "ragged": 1, "kv_lo": 9,
         "kv_hi": 16384, "page": 16, "format": "bf16", "dtype": "bf16", "mask": "causal", "window": 0, **heads},
        # token trees verified over an int8 cache
        {"name": "attend_tree_int8", "op": "attend", "n_seq": 16, "q": 31, "ragged": 1, "kv_lo": 31,
         "kv_hi": 16384, "page": 32, "format": "int8", "dtype": "f16", "mask": "tree", "window": 0, **heads},
        # a prompt chunk late in a long context
        {"name": "attend_chunk_long", "op": "attend", "n_seq": 1, "q": 2048, "ragged": 0, "kv_lo": 32768,
         "kv_hi": 32768, "page": 64, "format": "bf16", "dtype": "bf16", "mask": "causal", "window": 0, **heads},
        # chunks and single tokens in one call, sliding window, e4m3 pages
        {"name": "attend_mixed_window", "op": "attend", "n_seq": 16, "q": 1024, "ragged": 2, "kv_lo": 1024,
         "kv_hi": 8192, "page": 16, "format": "e4m3", "dtype": "bf16", "mask": "causal", "window": 2048, **heads},
        # a whole prompt from its first token, 64-wide heads
        {"name": "attend_prompt_64", "op": "attend", "n_seq": 2, "q": 4097, "ragged": 0, "kv_lo": 4097,
         "kv_hi": 4097, "page": 64, "format": "f16", "dtype": "f16", "mask": "causal", "window": 0,
         "heads": 32, "kv_heads": 8, "dim": 64},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 16), (28, 4), (40, 8)])
    c = {"op": rng.choice(["norm_rope", "append", "gather", "attend", "attend", "attend"]),
         "dtype": rng.choice(["f16", "bf16"]), "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128])}
    page = rng.choice([16, 32, 64, 128])
    rot = {"rotary": rng.choice([c["dim"], c["dim"], c["dim"] // 2, 48]), "layout": rng.choice(["half", "interleaved"]),
           "scaling": rng.choice(["none", "linear", "ntk", "yarn"])}
    fmt = rng.choice([c["dtype"], "int8", "e4m3"])
    if c["op"] == "norm_rope":
        return {**c, "dtype": rng.choice(["f16", "bf16", "f32"]), "rows": _log_int(rng, 1, 16384 if c["dim"] == 64 else 8192), **rot}
    if c["op"] == "append":
        n = _log_int(rng, 1, 64)
        q = _log_int(rng, 1, max(1, 32768 // n))
        read = rng.choice([0, 1]) if fmt != "int8" else 1
        return {**c, "n_seq": n, "q": q, "ragged": 1, "kv_lo": q, "kv_hi": q + _log_int(rng, 1, max(1, 65536 // n)),
                "page": page, "format": fmt, "fused": rng.choice([0, 1]), "read": read, **rot}
    if c["op"] == "gather":
        n = _log_int(rng, 1, 64)
        return {**c, "n_seq": n, "kv_lo": 1, "kv_hi": _log_int(rng, 1, 524288 // n), "page": page, "format": fmt}
    mask = rng.choice(["causal", "causal", "full", "tree"])
    q = _log_int(rng, 1, 40 if mask == "tree" else 2048)
    n = _log_int(rng, 1, max(1, min(64, 2048 // q)))
    kv = _log_int(rng, q, max(q, min(32768, 524288 // n, 16384 * 2048 // (n * q))))
    return {**c, "n_seq": n, "q": q, "ragged": rng.choice([0, 1, 2]), "kv_lo": q, "kv_hi": kv, "page": page,
            "format": fmt, "mask": mask, "window": rng.choice([0, 0, 0, 1 + kv // 3])}


# ---------------------------------------------------------------------------- lengths and frequencies

def _spread(n, lo, hi, turn):
    """n whole numbers over [lo, hi], the largest first, the others by the golden ratio."""
    return [hi if i == 0 else lo + int((i * 0.6180339887498949 + turn) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    n = case["n_seq"]
    kv = _spread(n, case["kv_lo"], case["kv_hi"], 0.0)
    if case["op"] == "gather":
        return kv, kv
    q = case["q"]
    if case["ragged"] == 0:
        new = [q] * n
    elif case["ragged"] == 1:                    # anything up to q
        new = _spread(n, 1, q, 0.35)
    else:                                        # one chunk in four, single tokens besides
        new = [max(1, q - 37 * i) if i % 4 == 0 else 1 for i in range(n)]
    return [min(a, b) for a, b in zip(new, kv)], kv


def _frequencies(case):
    """Angle per position of each rotated pair, and the factor on cosine and sine."""
    r, s = case["rotary"], 8.0
    i = [-2.0 * k / r for k in range(r // 2)]
    if case["scaling"] == "ntk":
        base = THETA * s ** (r / (r - 2))
        return [base ** x for x in i], 1.0
    f = [THETA ** x for x in i]
    if case["scaling"] == "linear":
        return [x / s for x in f], 1.0
    if case["scaling"] == "yarn":
        g = [min(1.0, max(0.0, (4096 * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
        return [(1 - a) * x / s + a * x for a, x in zip(g, f)], 0.1 * math.log(s) + 1.0
    return f, 1.0


# ---------------------------------------------------------------------------- inputs

def _pool(gen, n_pages, case, values):
    """One pool [n_pages, kv_heads, page, dim] in the case's format and its row scales."""
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    if not values:
        x = torch.zeros(shape, device="cuda", dtype=torch.float16)
    else:
        x = torch.randn(shape, device="cuda", dtype=torch.float16, generator=gen)
    if case["format"] in DTYPES:
        return x.to(DTYPES[case["format"]]), None
    if case["format"] == "int8":
        codes = (x * 36).clamp_(-127, 127).round_().to(torch.int8)
    else:
        codes = (x * 128).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scale = torch.rand(shape[:3], device="cuda", generator=gen) * 0.4 + 0.8
    return codes, scale / (36 if case["format"] == "int8" else 128) if values else scale * 0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, device="cuda", dtype=dt, generator=gen)

    s = {"case": case}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if "rotary" in case:
        s["freq"], s["magnitude"] = _frequencies(case)
        s["q_norm"], s["k_norm"] = (1 + 0.1 * torch.randn(dim, device="cuda", generator=gen) for _ in range(2))
    if case["op"] == "norm_rope":
        t = case["rows"]
        # projections of one matrix product: queries, keys and values of a token side by side
        qkv = randn(t, heads + 2 * kv_heads, dim)
        s["q"], s["k"] = qkv[:, :heads], qkv[:, heads:heads + kv_heads]
        first = int(torch.randint(0, 100000, (1,), generator=gen, device="cuda"))
        s["positions"] = torch.arange(first, first + t, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty(t, heads, dim, device="cuda", dtype=dt)
        s["k_out"] = torch.empty(t, kv_heads, dim, device="cuda", dtype=dt)
    else:
        new, kv = _lengths(case)
        per = -(-max(kv) // case["page"])
        used = [-(-x // case["page"]) for x in kv]
        n_pages = sum(used)
        order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
        pages = torch.full((len(kv), per), -1, dtype=torch.int32, device="cuda")
        slot = torch.arange(per, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]
        pages[slot] = order
        s["pages"] = pages
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["q_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        s["max_q"], s["max_kv"] = max(new), max(kv)
        t = sum(new)
        fill = case["op"] != "append"
        s["k_pool"], s["k_scale"] = _pool(gen, n_pages, case, fill)
        s["v_pool"], s["v_scale"] = _pool(gen, n_pages, case, fill)
        if case["op"] == "append":
            qkv = randn(t, heads + 2 * kv_heads, dim)
            s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
            s["q_out"] = torch.empty(t, heads, dim, device="cuda", dtype=dt)
        if case["op"] == "gather" or case.get("read"):
            s["k_rows"], s["v_rows"] = (torch.empty(t, kv_heads, dim, device="cuda", dtype=dt) for _ in range(2))
        if case["op"] == "attend":
            s["q"], s["o"] = randn(t, heads, dim), torch.empty(t, heads, dim, device="cuda", dtype=dt)
            if case["mask"] == "tree":
                # node j sees itself and a random part of the nodes before it
                i = torch.arange(t, device="cuda") - s["q_start"][_owner(s, t)]
                bits = torch.randint(0, 1 << 62, (t,), device="cuda", generator=gen)
                one = torch.ones_like(bits)
                s["tree"] = (bits & ((one << i) - 1)) | (one << i)
    if own:  # the handles over the cache, the batch and the rotation that a serving program keeps
        from speculative_decoding_draft_kv_gb300 import paged
        if "rotary" in case:
            s["rope"] = paged.PagedRope(case["rotary"], THETA, layout=case["layout"], scaling=case["scaling"],
                                        factor=8.0, original_len=4096)
        if "pages" in s:
            s["cache"] = paged.PagedCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
            s["batch"] = paged.PagedBatch(s["q_start"], s["kv_len"], s["pages"], s["max_q"], s["max_kv"])
        if case["op"] == "attend":
            n = paged.paged_attend_workspace(s["cache"], s["batch"], heads)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

def _owner(s, t):
    """The sequence of each row."""
    return torch.searchsorted(s["q_start"][1:].contiguous(), torch.arange(t, device="cuda", dtype=torch.int32),
                              right=True)


def _places(s, t):
    """Of each row: its position in the sequence, and the page and the row in it."""
    i = _owner(s, t)
    new = s["q_start"][1:] - s["q_start"][:-1]
    at = (s["kv_len"] - new - s["q_start"][:-1])[i] + torch.arange(t, device="cuda")
    page = s["case"]["page"]
    return at, s["pages"][i, at // page].long(), at % page


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _turn(s, x, positions, kind=torch.float32):
    """x [rows, heads, dim] turned by its positions."""
    r = s["case"]["rotary"]
    angle = positions.double()[:, None] * torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    cos, sin = ((f(angle) * s["magnitude"]).to(kind)[:, None] for f in (torch.cos, torch.sin))
    y = x.clone()
    if s["case"]["layout"] == "half":
        a, b = slice(0, r // 2), slice(r // 2, r)
    else:
        a, b = slice(0, r, 2), slice(1, r, 2)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _plain_norm_rope(s):
    q = _turn(s, _norm(s["q"].float(), s["q_norm"]), s["positions"])
    k = _turn(s, _norm(s["k"].float(), s["k_norm"]), s["positions"])
    return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype)}


def _quantise(x, fmt):
    top = x.abs().amax(-1, keepdim=True)
    y = x * torch.where(top > 1e-30, TOP[fmt] / top, 0.0)
    codes = y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return codes, (top / TOP[fmt])[..., 0]


def _put(pool, scales, rows, page, slot, fmt):
    """Rows [t, kv_heads, dim] into their places of the pool."""
    if fmt in DTYPES:
        pool[page, :, slot] = rows.to(pool.dtype)
        return
    codes, scale = _quantise(rows, fmt)
    pool.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
    scales[page, :, slot] = scale


def _rows(pool, scales, page, slot):
    """The values at some places, in 32 bits."""
    if scales is None:
        return pool[page, :, slot].float()
    return pool.view(torch.uint8)[page, :, slot].view(pool.dtype).float() * scales[page, :, slot][..., None]


def _written(s):
    """What an append changed or made, with codes as the values they stand for."""
    c = s["case"]
    out = {"q": s["q_out"]} if c["fused"] else {}
    if c["read"]:
        return {**out, "k": s["k_rows"], "v": s["v_rows"]}
    out |= {"k": s["k_pool"], "v": s["v_pool"]}
    return out if s["k_scale"] is None else {**out, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_append(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    at, page, slot = _places(s, k.shape[0])
    if c["fused"]:
        k = _turn(s, _norm(k, s["k_norm"]), at)
        s["q_out"].copy_(_turn(s, _norm(s["q"].float(), s["q_norm"]), at))
    _put(s["k_pool"], s["k_scale"], k, page, slot, c["format"])
    _put(s["v_pool"], s["v_scale"], v, page, slot, c["format"])
    if c["read"]:
        _plain_gather(s)
    return _written(s)


def _plain_gather(s):
    _, page, slot = _places(s, s["k_rows"].shape[0])
    s["k_rows"].copy_(_rows(s["k_pool"], s["k_scale"], page, slot))
    s["v_rows"].copy_(_rows(s["v_pool"], s["v_scale"], page, slot))
    return {"k": s["k_rows"], "v": s["v_rows"]}


def _visible(s, kind=None):
    """Truth values [n_seq, max_q, max_kv]: the positions that each new token sees."""
    c = s["case"]
    new = (s["q_start"][1:] - s["q_start"][:-1])[:, None, None]
    kv = s["kv_len"][:, None, None]
    i = torch.arange(s["max_q"], device="cuda")[None, :, None]
    p = torch.arange(s["max_kv"], device="cuda")[None, None]
    context = kv - new
    if c["mask"] == "causal":
        see = p <= context + i
        low = context + i - c["window"] + 1
    else:
        see = p < kv
        low = context - c["window"]
        if c["mask"] == "tree":
            word = s["tree"][(s["q_start"][:-1, None, None] + i).clamp(max=s["tree"].numel() - 1)]
            see = (p < context) | (see & ((word >> (p - context).clamp(0, 62)) & 1).bool())
    if c["window"]:
        see = see & (p >= low)
    return see & (i < new)


def _plain_attend(s):
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    page = c["page"]
    n, lq, lk = s["kv_len"].numel(), s["max_q"], s["max_kv"]
    p = torch.arange(lk, device="cuda")
    pages = s["pages"][:, p // page].clamp(min=0).long()
    slot = (p % page)[None].expand(n, lk)
    alive = (p[None] < s["kv_len"][:, None])[..., None, None]
    k, v = (torch.where(alive, _rows(s[a + "_pool"], s[a + "_scale"], pages, slot), 0.0).permute(0, 2, 1, 3)
            for a in "kv")
    row = s["q_start"][:-1, None] + torch.arange(lq, device="cuda")
    row = row.clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][row].float().view(n, lq, c["kv_heads"], group, c["dim"])
    q = q.permute(0, 2, 3, 1, 4).reshape(n, c["kv_heads"], group * lq, c["dim"])
    see = _visible(s)[:, None, None]
    score = (q @ k.transpose(2, 3)).view(n, c["kv_heads"], group, lq, lk).mul_(c["dim"] ** -0.5)
    score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    o = (score.view(n, c["kv_heads"], group * lq, lk) @ v).view(n, c["kv_heads"], group, lq, c["dim"])
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, lq, c["heads"], c["dim"])
    t = s["o"].shape[0]
    i = _owner(s, t)
    s["o"].copy_(o[i, torch.arange(t, device="cuda") - s["q_start"][i]])
    return {"o": s["o"]}


def run(state):
    c = state["case"]
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "gather": _plain_gather,
            "attend": _plain_attend}[c["op"]](state)


def _own(s):
    from speculative_decoding_draft_kv_gb300 import paged
    c = s["case"]
    if c["op"] == "attend":
        paged.paged_attend(s["cache"], s["batch"], s["q"], s["o"], mask=c["mask"], window=c["window"],
                           tree=s.get("tree"), workspace=s["workspace"])
        return {"o": s["o"]}
    if c["op"] == "gather":
        paged.paged_gather(s["cache"], s["batch"], s["k_rows"], s["v_rows"])
        return {"k": s["k_rows"], "v": s["v_rows"]}
    if c["op"] == "norm_rope":
        paged.paged_norm_rope(s["positions"], s["rope"], EPS, q=s["q"], q_norm=s["q_norm"], q_out=s["q_out"],
                              k=s["k"], k_norm=s["k_norm"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["fused"]:
        paged.paged_append(s["cache"], s["batch"], s["k"], s["v"], rope=s["rope"], eps=EPS, k_norm=s["k_norm"],
                           q=s["q"], q_norm=s["q_norm"], q_out=s["q_out"])
    else:
        paged.paged_append(s["cache"], s["batch"], s["k"], s["v"])
    if c["read"]:
        paged.paged_gather(s["cache"], s["batch"], s["k_rows"], s["v_rows"])
    return _written(s)


# ---------------------------------------------------------------------------- work

def work(case):
    d, h, g = case["dim"], case["heads"], case["kv_heads"]
    wide = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm_rope":
        values = case["rows"] * (h + g) * d
        return {"bytes": 2 * wide * values + 4 * case["rows"], "flops": 8 * values}
    row = 2 * g * (2 * d if case["format"] in DTYPES else d + 4)         # K and V of one token in the cache
    new, kv = _lengths(case)
    t = sum(new)
    if case["op"] == "gather":
        return {"bytes": t * (row + 2 * g * d * wide), "flops": 2 * t * g * d}
    if case["op"] == "append":
        b = t * (row + 2 * g * d * wide)
        if case["fused"]:
            b += 2 * t * h * d * wide
        if case["read"]:
            b += t * (row + 2 * g * d * wide)
        return {"bytes": b, "flops": 8 * t * (2 * g + (h if case["fused"] else 0)) * d}
    w, pairs, rows = case["window"], 0, 0
    for n, l in zip(new, kv):
        c = l - n
        if case["mask"] == "causal":
            # token i sees c + i + 1 positions, the last w of them under a window
            full = n if not w else min(n, max(0, w - c))
            pairs += full * c + full * (full + 1) // 2 + (n - full) * w
            rows += l if not w else min(l, w + n - 1)
        else:
            seen = c if not w else min(c, w)
            own_pairs = n * n if case["mask"] == "full" else n * (n + 3) // 4
            pairs += n * seen + own_pairs
            rows += seen + n
    return {"bytes": rows * row + 2 * t * h * d * wide, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------- 64 bits

def _exact_rope(x, positions, w, freq, magnitude, case):
    """From the definition: every pair as one complex number."""
    x = x.double()
    x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    r = case["rotary"]
    a = positions.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(a, magnitude), a)
    head, rest = x[..., :r], x[..., r:]
    if case["layout"] == "half":
        z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    return torch.cat([head, rest], -1)


def _exact_codes(x, fmt):
    scale = x.abs().amax(-1) / TOP[fmt]
    y = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    return (y.round() if fmt == "int8" else y.float().to(torch.float8_e4m3fn).double()), scale


def _exact_rows(pool, scale, ids, page, length):
    """One sequence's cached rows [length, kv_heads, dim], page after page."""
    x = pool[ids.long().clamp(min=0)] if scale is None else (
        pool.view(torch.uint8)[ids.long().clamp(min=0)].view(pool.dtype))
    x = x.double()
    if scale is not None:
        x = x * scale[ids.long().clamp(min=0)].double()[..., None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:length]


def exact(case, seed):
    if work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return {a: _exact_rope(s[a], s["positions"], s[a + "_norm"], s["freq"], s["magnitude"], case) for a in "qk"}
    new, kv = _lengths(case)
    out, at = {}, 0
    if case["op"] == "gather":
        for a in "kv":
            out[a] = torch.cat([_exact_rows(s[a + "_pool"], s[a + "_scale"], s["pages"][i], case["page"], l)
                                for i, l in enumerate(kv)])
        return out
    if case["op"] == "append":
        where = torch.cat([torch.arange(l - n, l, device="cuda") for n, l in zip(new, kv)])
        x = {a: s[a].double() for a in "kv"}
        if case["fused"]:
            x["k"] = _exact_rope(s["k"], where, s["k_norm"], s["freq"], s["magnitude"], case)
            out["q"] = _exact_rope(s["q"], where, s["q_norm"], s["freq"], s["magnitude"], case)
        for a in "kv":
            codes, scale = (x[a], None) if case["format"] in DTYPES else _exact_codes(x[a], case["format"])
            if case["read"]:
                out[a] = codes if scale is None else codes * scale[..., None]
                continue
            pool = s[a + "_pool"].double()
            scales = None if scale is None else s[a + "_scale"].double()
            for i, (n, l) in enumerate(zip(new, kv)):
                pos = torch.arange(l - n, l, device="cuda")
                ids = s["pages"][i][pos // case["page"]].long()
                pool[ids, :, pos % case["page"]] = codes[at:at + n]
                if scales is not None:
                    scales[ids, :, pos % case["page"]] = scale[at:at + n]
                at += n
            at = 0
            out[a] = pool
            if scales is not None:
                out[a + "_scale"] = scales
        return out
    group = case["heads"] // case["kv_heads"]
    parts = []
    for i, (n, l) in enumerate(zip(new, kv)):
        k, v = (_exact_rows(s[a + "_pool"], s[a + "_scale"], s["pages"][i], case["page"], l) for a in "kv")
        q = s["q"][at:at + n].double()
        c = l - n
        pos = torch.arange(l, device="cuda")
        tok = torch.arange(n, device="cuda")[:, None]
        if case["mask"] == "causal":
            hidden = pos > c + tok
            if case["window"]:
                hidden = hidden | (c + tok - pos >= case["window"])
        else:
            hidden = torch.zeros(n, l, dtype=torch.bool, device="cuda")
            if case["window"]:
                hidden[:, :max(0, c - case["window"])] = True
            if case["mask"] == "tree":
                word = s["tree"][at:at + n, None]
                hidden[:, c:] = ((word >> torch.arange(n, device="cuda")) & 1) == 0
        o = torch.empty(n, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        for j in range(case["heads"]):
            z = (q[:, j] @ k[:, j // group].T) / math.sqrt(case["dim"])
            p = torch.softmax(z.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0)
            o[:, j] = p @ v[:, j // group]
        parts.append(o)
        at += n
    return {"o": torch.cat(parts)}
