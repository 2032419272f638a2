"""The paged 4-bit key/value cache operators as a serving loop calls them: what is measured, their plain forms, and
their values in 64 bits.

`own = False` computes with elementary torch operations in 32 bits; `own = True` calls the library. Kinds of cases:

  plan    block tables, slot maps, positions and query offsets of one step from the requests' lengths
  append  the step's new key / value rows quantized into their cache slots, then read back as values
  attend  attention of the step's queries over the 4-bit cache (one token, a few tokens, or long chunks per request)
  step    plan, append and attend in sequence: one layer of one decoding step

A case gives sizes and head layout; the lengths follow from it by a fixed low-discrepancy sequence (their order, the
pages and all values come from the seed), so the work of a case does not depend on the seed.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_GOLDEN = 0.6180339887498949


def listed():
    a = {"kind": "attend", "window": 0}
    return [
        # bookkeeping of a decoding step of 64 running requests
        {"name": "plan_decode_64", "kind": "plan", "batch": 64, "q_min": 1, "q_max": 1, "kv_min": 0, "kv_max": 8192,
         "finished": 0, "page": 64},
        # bookkeeping of a large step: prompts being read, waiting and finished requests among them, small pages
        {"name": "plan_mixed_1000", "kind": "plan", "batch": 1000, "q_min": 0, "q_max": 133, "kv_min": 0,
         "kv_max": 5000, "finished": 37, "page": 16},
        # new rows of a decoding step
        {"name": "append_decode_64", "kind": "append", "tokens": 64, "hkv": 8, "d": 128, "gs": 64, "page": 64,
         "dtype": "bf16"},
        # new rows of a long prompt step, finer groups, an odd number of tokens
        {"name": "append_prompt_20011", "kind": "append", "tokens": 20011, "hkv": 8, "d": 128, "gs": 32, "page": 32,
         "dtype": "f16"},
        # one request, one token, a short context: nothing but latency
        {**a, "name": "decode_1x300", "batch": 1, "q_min": 1, "q_max": 1, "kv_min": 300, "kv_max": 300, "hkv": 8,
         "g": 4, "d": 128, "gs": 64, "page": 64, "dtype": "bf16"},
        # an ordinary decoding batch with ragged contexts
        {**a, "name": "decode_48x4500", "batch": 48, "q_min": 1, "q_max": 1, "kv_min": 37, "kv_max": 4500, "hkv": 8,
         "g": 4, "d": 128, "gs": 64, "page": 64, "dtype": "bf16"},
        # few requests with very long contexts
        {**a, "name": "decode_4x131072", "batch": 4, "q_min": 1, "q_max": 1, "kv_min": 90001, "kv_max": 131072,
         "hkv": 8, "g": 8, "d": 128, "gs": 64, "page": 128, "dtype": "f16"},
        # 32-bit activations, small heads and groups, an odd number of query heads per key head
        {**a, "name": "decode_f32_d64", "batch": 30, "q_min": 1, "q_max": 1, "kv_min": 1, "kv_max": 6000, "hkv": 4,
         "g": 7, "d": 64, "gs": 32, "page": 16, "dtype": "f32"},
        # several tokens per request checked at once, sliding window, one key head for each of 16 query heads
        {**a, "name": "verify_20x16k_window", "batch": 20, "q_min": 2, "q_max": 6, "kv_min": 500, "kv_max": 16000,
         "hkv": 2, "g": 16, "d": 128, "gs": 128, "page": 32, "dtype": "f16", "window": 4096},
        # prompt chunks of several requests on top of what they have in the cache
        {**a, "name": "chunk_6x1500", "batch": 6, "q_min": 333, "q_max": 1500, "kv_min": 1500, "kv_max": 7000,
         "hkv": 4, "g": 8, "d": 128, "gs": 64, "page": 64, "dtype": "bf16"},
        # one whole long prompt
        {**a, "name": "prompt_1x8192", "batch": 1, "q_min": 8192, "q_max": 8192, "kv_min": 8192, "kv_max": 8192,
         "hkv": 8, "g": 4, "d": 128, "gs": 64, "page": 64, "dtype": "bf16"},
        # one layer of a decoding step: lengths to slots, rows into the cache, attention
        {"name": "step_96x2000", "kind": "step", "batch": 96, "q_min": 1, "q_max": 1, "kv_min": 20, "kv_max": 2000,
         "hkv": 8, "g": 4, "d": 128, "gs": 64, "page": 64, "dtype": "bf16", "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "append", "decode", "decode", "decode", "verify", "chunk", "chunk", "step"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "plan":
        q_max = _log(rng, 1, 130)
        return {"kind": "plan", "batch": _log(rng, 1, 1000), "q_min": rng.randint(0, 1), "q_max": q_max, "kv_min": 0,
                "kv_max": _log(rng, 16, 8192), "finished": rng.choice([0, 0, 3, 11]), "page": page}
    d = rng.choice([64, 128, 128])
    c = {"hkv": rng.choice([1, 2, 4, 8]), "d": d, "gs": rng.choice([g for g in (32, 64, 128) if g <= d]), "page": page}
    if kind == "append":
        return {"kind": "append", "tokens": _log(rng, 1, 20000), **c, "dtype": rng.choice(["bf16", "f16", "f32"])}
    c["g"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    if kind in ("decode", "verify", "step"):
        batch = _log(rng, 1, 200)
        kv_max = _log(rng, 16, max(17, min(131072, 3000000 // (batch * c["hkv"]))))
        kv_min = rng.choice([1, max(1, kv_max // 3), kv_max])
        q = (1, 1) if kind != "verify" else (1, rng.randint(2, 8))
        return {"kind": "step" if kind == "step" else "attend", "batch": batch, "q_min": q[0], "q_max": q[1],
                "kv_min": max(kv_min, q[1]), "kv_max": max(kv_max, q[1]), **c, "window": window,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f16", "f32"])}
    batch = _log(rng, 1, 8)
    heads = c["hkv"] * c["g"]
    kv_max = _log(rng, 300, 8192)
    # scores of the plain form: batch * heads * q * kv values of 4 bytes
    q_max = max(9, min(kv_max, 2000000000 // (batch * heads * kv_max)))
    q_max = _log(rng, 9, max(10, q_max))
    return {"kind": "attend", "batch": batch, "q_min": max(1, q_max // rng.choice([1, 2, 9])), "q_max": q_max,
            "kv_min": max(q_max, kv_max // 2), "kv_max": max(kv_max, q_max), **c, "window": window,
            "dtype": rng.choice(["bf16", "f16"])}


# ---------------------------------------------------------------- lengths

def _spread(n, lo, hi, phase):
    """n lengths between lo and hi (both met when n > 1 and they differ)."""
    v = [lo + int((hi - lo + 1) * ((phase + i * _GOLDEN) % 1.0)) for i in range(n)]
    v = [min(x, hi) for x in v]
    if n > 1:
        v[0], v[n // 2] = hi, lo
    elif n == 1:
        v[0] = hi
    return v


def _lengths(case):
    """(new tokens, cached tokens before the step) of each request. For `attend` the second is what the cache holds
    with the new tokens among them."""
    n = case["batch"]
    q = _spread(n, case["q_min"], case["q_max"], 0.25)
    kv = _spread(n, case["kv_min"], case["kv_max"], 0.6)
    for i in range(case.get("finished", 0)):
        q[(i * 7 + 3) % n] = -1
    return q, kv


def _pairs(case):
    """(query, key) pairs that the causal mask and the window leave, over all requests; keys that some query sees."""
    pairs = keys = 0
    q, kv = _lengths(case)
    add = 1 if case["kind"] == "step" else 0
    w = case["window"]
    for a, b in zip(q, kv):
        b += a * add
        if w:
            n = sum(min(w, b - a + i + 1) for i in range(a))
            keys += min(b, w + a - 1)
        else:
            n = a * (b - a) + a * (a + 1) // 2
            keys += b
        pairs += n
    return pairs, keys


def work(case):
    if case["kind"] == "plan":
        q, kv = _lengths(case)
        p = case["page"]
        new = sum(max(x, 0) for x in q)
        touched = sum(-(-(b + a) // p) - -(-b // p) if a >= 0 else -(-b // p) for a, b in zip(q, kv))
        return {"bytes": 16 * len(q) + 12 * new + 8 * touched, "flops": 0}
    e = 4 if case["dtype"] == "f32" else 2
    row = case["d"] // 2 + 2 * e * (case["d"] // case["gs"])    # a cached row of one head: codes, scales and biases
    if case["kind"] == "append":
        n = case["tokens"] * case["hkv"] * 2
        return {"bytes": n * (case["d"] * e + 2 * row + 4 * case["d"]) + 8 * case["tokens"], "flops": 4 * n * case["d"]}
    pairs, keys = _pairs(case)
    q, _ = _lengths(case)
    heads = case["hkv"] * case["g"]
    n = sum(q)
    by = 2 * keys * case["hkv"] * row + 2 * n * heads * case["d"] * e
    if case["kind"] == "step":
        by += n * case["hkv"] * 2 * (case["d"] * e + row) + 16 * n
    return {"bytes": by, "flops": 4 * pairs * heads * case["d"]}


# ---------------------------------------------------------------- inputs

def _quantize(x, gs, dt):
    """x [..., D] float32 -> (packed int32 [..., D/8], scales, biases [..., D/gs] in dt): per group the bias is the
    least value, the scale a fifteenth of the range, both rounded to dt before the codes are taken."""
    g = x.unflatten(-1, (-1, gs))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / torch.full((), 15.0, device=x.device)).to(dt)
    b = lo.to(dt)
    sf = s.float().unsqueeze(-1)
    q = ((g - b.float().unsqueeze(-1)) / torch.where(sf == 0, 1.0, sf)).round().clamp(0, 15)
    q = torch.where(sf == 0, 0.0, q).long().flatten(-2).unflatten(-1, (-1, 8))
    w = (q << torch.arange(0, 32, 4, device=x.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int(), s, b


def _codes(w):
    """[..., W] int32 words -> [..., 8 W] codes in float32, low nibble first."""
    return ((w.unsqueeze(-1) >> torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)) & 15).flatten(-2).float()


def _values(w, s, b, gs):
    """What packed rows stand for, float32 [..., D]."""
    q = _codes(w).unflatten(-1, (-1, gs))
    return (s.float().unsqueeze(-1) * q + b.float().unsqueeze(-1)).flatten(-2)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _pool(case, blocks, gen, outliers):
    """A cache of `blocks` pages, all filled with quantized rows: unit values with a few large channels, as keys have
    (used pages and pages that other requests left behind look alike)."""
    shape = (blocks, case["hkv"], case["page"], case["d"])
    dt = _DT[case["dtype"]]
    packed = torch.empty(shape[:-1] + (case["d"] // 8,), dtype=torch.int32, device="cuda")
    scales = torch.empty(shape[:-1] + (case["d"] // case["gs"],), dtype=dt, device="cuda")
    biases = torch.empty_like(scales)
    gain = torch.ones(case["hkv"], 1, case["d"], device="cuda")
    if outliers:
        gain[:, :, torch.randint(case["d"], (3,), generator=gen, device="cuda")] = 4.0
    n = max(1, (1 << 27) // (case["hkv"] * case["page"] * case["d"]))
    for i in range(0, blocks, n):
        x = torch.randn((min(n, blocks - i),) + shape[1:], generator=gen, device="cuda") * gain
        packed[i:i + n], scales[i:i + n], biases[i:i + n] = _quantize(x, case["gs"], dt)
    return packed, scales, biases


def _ints(v, dt=torch.int32):
    return torch.tensor(v, dtype=dt).cuda()


def prepare(case, seed):
    gen = _gen(seed)
    host = torch.Generator().manual_seed(seed * 104729 + 7)
    page = case["page"]
    st = {"case": case}
    if case["kind"] == "append":
        n = case["tokens"]
        blocks = -(-n // page) + 5
        dt = _DT[case["dtype"]]
        # key and value rows as slices of one projection's output
        qkv = torch.randn(n, case["hkv"] * 2 + 2, case["d"], generator=gen, device="cuda").to(dt)
        st["k"], st["v"] = qkv[:, 2:2 + case["hkv"]], qkv[:, 2 + case["hkv"]:]
        perm = torch.randperm(blocks, generator=host)
        t = torch.arange(n)
        st["slots"] = (perm[t // page] * page + t % page).cuda()
        st["k_cache"], st["v_cache"] = _pool(case, blocks, gen, False), _pool(case, blocks, gen, False)
        return st

    q, kv = _lengths(case)
    order = torch.randperm(case["batch"], generator=host).tolist()
    q, kv = [q[i] for i in order], [kv[i] for i in order]
    if case["kind"] == "attend":
        kv = [max(a, b) for a, b in zip(q, kv)]
        total = kv
    else:
        total = [b + max(a, 0) for a, b in zip(q, kv)]
    held = kv if case["kind"] != "attend" else total
    width = max(1, max(-(-t // page) for t in total))
    have = [-(-h // page) for h in held]
    need = sum(-(-t // page) for t in total)
    blocks = need + 7
    perm = torch.randperm(blocks, generator=host)
    rows = torch.full((case["batch"], width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(have):
        rows[i, :n] = perm[at:at + n].int()
        at += n
    st["table"] = rows.cuda()
    st["tokens"] = sum(max(a, 0) for a in q)
    if case["kind"] in ("plan", "step"):
        st["free"] = torch.zeros(blocks, dtype=torch.int32)
        st["free"][:blocks - at] = perm[at:].int()
        st["free"] = st["free"].cuda()
        st["free_count"] = _ints([blocks - at])
        st["q_lens"], st["kv_lens"] = _ints(q), _ints(kv)
        if case["kind"] == "plan":
            return st
    else:
        st["kv_lens"] = _ints(total)
        st["cu_q"] = _ints([sum(q[:i]) for i in range(len(q) + 1)])
    dt = _DT[case["dtype"]]
    heads = case["hkv"] * case["g"]
    qkv = torch.randn(st["tokens"], heads + 2 * case["hkv"], case["d"], generator=gen, device="cuda").to(dt)
    st["q"], st["k"], st["v"] = qkv.split([heads, case["hkv"], case["hkv"]], 1)
    st["k_cache"], st["v_cache"] = _pool(case, blocks, gen, True), _pool(case, blocks, gen, False)
    st["scale"] = case["d"] ** -0.5
    st["max_q"] = max(q)
    return st


# ---------------------------------------------------------------- plain forms

def _plan(st):
    """Releases the pages of finished requests (new length -1) onto the stack of free pages, takes the pages that the
    new tokens need from its top, and lists where each new token goes."""
    page = st["case"]["page"]
    q, kv, table, count = st["q_lens"].long(), st["kv_lens"].long(), st["table"], st["free_count"].long()
    dev = q.device
    done = q < 0
    had = (kv + page - 1) // page
    new = torch.where(done, 0, q)
    now = torch.where(done, 0, kv + new)
    gave = torch.where(done, had, 0)
    took = torch.where(done, 0, (now + page - 1) // page - had)
    gave_to, took_to = gave.cumsum(0), took.cumsum(0)
    col = torch.arange(table.shape[1], device=dev)
    # stack of free pages: finished requests' pages on top of what was there
    put = col[None, :] < gave[:, None]
    at = torch.where(put, count + (gave_to - gave)[:, None] + col, st["free"].shape[0])
    free = torch.cat([st["free"], st["free"].new_zeros(1)])
    free.scatter_(0, at.flatten(), table.flatten())
    top = count + gave_to[-1:]
    get = (col[None, :] >= had[:, None]) & (col[None, :] < (had + took)[:, None])
    i = top - 1 - ((took_to - took - had)[:, None] + col)
    table = torch.where(get, free[torch.where(get, i, 0)], table)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(st["tokens"], device=dev)
    r = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[r] + t - cu[r]
    slots = table[r, pos // page].long() * page + pos % page
    return {"block_table": table, "slots": slots, "positions": pos.int(), "cu_q": cu.int(), "kv_lens": now.int(),
            "free_blocks": free[:-1], "free_count": (top - took_to[-1:]).int()}


def _append(st, slots):
    page, gs = st["case"]["page"], st["case"]["gs"]
    for x, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        for part, to in zip(_quantize(x.float(), gs, x.dtype), cache):
            to[slots // page, :, slots % page] = part


def _read(st):
    page, gs = st["case"]["page"], st["case"]["gs"]
    p, o = st["slots"] // page, st["slots"] % page
    return [_values(*(c[p, :, o] for c in cache), gs) for cache in (st["k_cache"], st["v_cache"])]


def _attend(st, table, kv_lens, cu):
    c = st["case"]
    hkv, g, d, page = c["hkv"], c["g"], c["d"], c["page"]
    q, n, longest = st["q"], st["tokens"], st["max_q"]
    dev = q.device
    b = kv_lens.shape[0]
    kv_lens, cu = kv_lens.long(), cu.long()
    lens = cu[1:] - cu[:-1]
    idx = table.clamp(min=0).long()
    # [b, hkv, keys, d]
    k, v = (_values(*(x[idx].transpose(1, 2).flatten(2, 3) for x in cache), c["gs"])
            for cache in (st["k_cache"], st["v_cache"]))
    at = (cu[:-1, None] + torch.arange(longest, device=dev)).clamp(max=n - 1)
    qp = q.float()[at].unflatten(2, (hkv, g)).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * longest, d)
    s = (qp @ k.transpose(2, 3)).mul_(st["scale"]).unflatten(2, (g, longest))
    pos = (kv_lens - lens)[:, None] + torch.arange(longest, device=dev)
    key = torch.arange(k.shape[2], device=dev)
    see = key <= pos[:, :, None]
    if c["window"]:
        see &= key > (pos - c["window"])[:, :, None]
    see &= key < kv_lens[:, None, None]
    see = see[:, None, None]
    s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((key < kv_lens[:, None])[:, None, :, None], v, 0.0)
    o = (p.flatten(2, 3) @ v).unflatten(2, (g, longest)) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, longest, hkv * g, d)
    t = torch.arange(n, device=dev)
    r = torch.searchsorted(cu, t, right=True) - 1
    return o[r, t - cu[r]].to(q.dtype)


def run(st):
    c = st["case"]
    if own:
        return _run_own(st)
    if c["kind"] == "plan":
        return _plan(st)
    if c["kind"] == "append":
        _append(st, st["slots"])
        return _read(st)
    if c["kind"] == "attend":
        return _attend(st, st["table"], st["kv_lens"], st["cu_q"])
    p = _plan(st)
    _append(st, p["slots"])
    return {"out": _attend(st, p["block_table"], p["kv_lens"], p["cu_q"]), **p}


def _run_own(st):
    import gemm_affine_int4_gb300 as g4
    c = st["case"]
    if c["kind"] in ("plan", "step"):
        p = g4.gai4_kv_plan(st["kv_lens"], st["q_lens"], st["table"], st["free"], st["free_count"], c["page"],
                            st["tokens"])
        plan = {"block_table": st["table"], "slots": p.slots, "positions": p.positions, "cu_q": p.cu_q,
                "kv_lens": p.kv_lens, "free_blocks": st["free"], "free_count": p.free_count}
        if c["kind"] == "plan":
            return plan
        slots, kv_lens, cu_q = p.slots, p.kv_lens, p.cu_q
    elif c["kind"] == "append":
        slots = st["slots"]
    else:
        kv_lens, cu_q = st["kv_lens"], st["cu_q"]
    if c["kind"] in ("append", "step"):
        g4.gai4_kv_append(st["k"], st["v"], slots, st["k_cache"], st["v_cache"], group_size=c["gs"])
        if c["kind"] == "append":
            return [g4.gai4_kv_read(cache, slots, group_size=c["gs"]) for cache in (st["k_cache"], st["v_cache"])]
    out = g4.gai4_kv_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], kv_lens, cu_q, group_size=c["gs"],
                               scale=st["scale"], window=c["window"], max_q_len=st["max_q"])
    return out if c["kind"] == "attend" else {"out": out, **plan}


# ---------------------------------------------------------------- values in 64 bits

def _exact_values(cache, pages, offs, gs):
    """Rows (pages, offs) of a cache as float64 [rows, hkv, d]."""
    packed, scales, biases = cache
    w = packed[pages, :, offs].long() & 0xFFFFFFFF
    code = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], -1).reshape(w.shape[0], w.shape[1], -1).double()
    s = scales[pages, :, offs].double().repeat_interleave(gs, -1)
    b = biases[pages, :, offs].double().repeat_interleave(gs, -1)
    return s * code + b


def _exact_attend(st, table, kv_lens, cu):
    c = st["case"]
    page, g, w = c["page"], c["g"], c["window"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for r in range(len(kv_lens)):
        n, first, last = kv_lens[r], cu[r], cu[r + 1]
        lo = max(0, n - (last - first) - w + 1) if w else 0
        if n <= 0 or first == last:
            continue
        j = torch.arange(lo, n, device="cuda")
        pages, offs = table[r][j // page].long(), j % page
        k, v = (_exact_values(x, pages, offs, c["gs"]) for x in (st["k_cache"], st["v_cache"]))
        for h in range(c["hkv"]):
            kh, vh = k[:, h].contiguous(), v[:, h].contiguous()
            step = max(1, (1 << 27) // (g * (n - lo)))
            for t in range(first, last, step):
                e = min(last, t + step)
                s = torch.einsum("tgd,kd->tgk", st["q"][t:e, h * g:(h + 1) * g].double(), kh) * st["scale"]
                pos = torch.arange(t - first, e - first, device="cuda")[:, None] + (n - (last - first))
                hide = (j > pos) | ((j <= pos - w) if w else torch.zeros_like(j > pos))
                s = s.masked_fill(hide[:, None], -math.inf)
                out[t:e, h * g:(h + 1) * g] = torch.softmax(s, -1).nan_to_num(0.0) @ vh
    return out


def exact(case, seed):
    if case["kind"] == "plan":
        return None
    st = prepare(case, seed)
    if case["kind"] == "attend":
        return _exact_attend(st, st["table"], st["kv_lens"].tolist(), st["cu_q"].tolist())
    # the codes are defined by rounded 32-bit steps, and so are what the cache holds after them
    if case["kind"] == "append":
        outs = []
        for x, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
            rows = torch.arange(case["tokens"], device="cuda")
            parts = [p.unsqueeze(2) for p in _quantize(x.float(), case["gs"], x.dtype)]
            outs.append(_exact_values(parts, rows, torch.zeros_like(rows), case["gs"]))
        return outs
    page = case["page"]
    q, kv, free, count = (st[k].tolist() for k in ("q_lens", "kv_lens", "free", "free_count"))
    table, n, cu, slots = st["table"].clone().cpu(), count[0], [0], []
    for r, (a, b) in enumerate(zip(q, kv)):
        for i in range(b, b + a):
            if i % page == 0:
                n -= 1
                table[r, i // page] = free[n]
            slots.append(int(table[r, i // page]) * page + i % page)
        cu.append(cu[-1] + a)
    at = _ints(slots, torch.int64)
    for x, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        for part, to in zip(_quantize(x.float(), case["gs"], x.dtype), cache):
            to[at // page, :, at % page] = part
    return {"out": _exact_attend(st, table.cuda(), [a + b for a, b in zip(q, kv)], cu)}
