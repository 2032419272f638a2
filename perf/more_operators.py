"""The operators of a layer around the attention, as a serving loop calls them: what is measured, their plain forms, and
their values in 64 bits.

`own = False` computes with elementary torch operations in 32 bits; `own = True` calls the library. Kinds of cases:

  rope     rotary positions of the step's query and key rows
  norm     root-mean-square norm, with the residual's addition, and rows in 8-bit floating point with their scales
  quant_x  activations into e4m3 with a scale for each 128 elements of a row
  quant_w  weights into e4m3 with a scale for each block of 128 x 128
  mm       the product of such activations with such weights
  layer    norm, product, rotary positions, quantization and product in sequence: a layer without its attention

A case gives sizes and types; all values come from the seed.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_GROUP = 128


def listed():
    return [
        # query and key rows of a decoding step: far positions, nothing but latency
        {"name": "rope_decode_64", "kind": "rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "far": 8192, "dtype": "bf16"},
        # a long prompt, adjacent pairs, positions stretched to a long context, an odd number of tokens
        {"name": "rope_prompt_20011", "kind": "rope", "tokens": 20011, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": True, "scaling": "yarn", "far": 131072, "dtype": "f16"},
        # 32-bit activations, small heads of which a part is rotated, very far positions
        {"name": "rope_f32_part", "kind": "rope", "tokens": 4099, "hq": 28, "hkv": 4, "d": 80, "rot": 32,
         "interleaved": False, "scaling": "linear", "far": 4000000, "dtype": "f32"},
        # the norm before a product of a decoding step
        {"name": "norm_decode_64", "kind": "norm", "rows": 64, "cols": 4096, "residual": True, "fp8": True,
         "dtype": "bf16"},
        # the same of a long prompt
        {"name": "norm_prompt_20011", "kind": "norm", "rows": 20011, "cols": 5120, "residual": True, "fp8": True,
         "dtype": "bf16"},
        # activations of a small batch before a product
        {"name": "quant_x_33", "kind": "quant_x", "rows": 33, "cols": 14336, "dtype": "f16"},
        # a layer's weights, once when they are loaded
        {"name": "quant_w_14336x5120", "kind": "quant_w", "rows": 14336, "cols": 5120, "dtype": "f32"},
        # one token: the weights are read once and that is all
        {"name": "mm_1x4096x4096", "kind": "mm", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a decoding batch
        {"name": "mm_56x5120x17408", "kind": "mm", "m": 56, "n": 5120, "k": 17408, "dtype": "bf16"},
        # a prompt chunk, sizes that end inside tiles and blocks
        {"name": "mm_1111x5000x14416", "kind": "mm", "m": 1111, "n": 5000, "k": 14416, "dtype": "f16"},
        # a long prompt
        {"name": "mm_8192x14336x5120", "kind": "mm", "m": 8192, "n": 14336, "k": 5120, "dtype": "bf16"},
        # a layer of a decoding step
        {"name": "layer_48", "kind": "layer", "tokens": 48, "hidden": 4096, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "far": 8192, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "norm", "norm", "quant_x", "quant_w", "mm", "mm", "mm", "mm", "layer"])
    dt = rng.choice(["bf16", "f16"] if kind == "layer" else ["bf16", "bf16", "f16", "f16", "f32"])
    if kind in ("rope", "layer"):
        d = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        c = {"hq": hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4]),
             "interleaved": rng.choice([False, True]), "scaling": rng.choice(["none", "linear", "ntk", "yarn", "smooth"]),
             "far": _log(rng, 100, 4000000)}
        if kind == "layer":
            return {"kind": kind, "tokens": _log(rng, 1, 2000), "hidden": 16 * _log(rng, 16, 400), **c, "dtype": dt}
        return {"kind": kind, "tokens": _log(rng, 1, min(20000, 100000000 // ((c["hq"] + hkv) * d))), **c, "dtype": dt}
    if kind == "mm":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 16384), 16 * _log(rng, 8, 1024)
        return {"kind": kind, "m": min(m, 600000000000 // (n * k)), "n": n, "k": k, "dtype": dt}
    cols = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 16, 2048), 128 * _log(rng, 1, 128)])
    rows = _log(rng, 1, min(20000, 73000000 // cols))
    if kind == "norm":
        return {"kind": kind, "rows": rows, "cols": cols, "residual": rng.choice([False, True]),
                "fp8": rng.choice([False, True, True]), "dtype": dt}
    return {"kind": kind, "rows": rows, "cols": cols, "dtype": dt}


def _blocks(n):
    return -(-n // _GROUP)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    kind = case["kind"]
    if kind == "rope":
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * rows * case["d"] * e + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * rows * case["rot"]}
    if kind == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * e + 4 * _blocks(k) * (m + _blocks(n)), "flops": 2 * m * n * k}
    if kind == "layer":
        t, h, o = case["tokens"], case["hidden"], case["hq"] * case["d"]
        n = o + 2 * case["hkv"] * case["d"]
        weights = n * h + h * o + 4 * (_blocks(n) * _blocks(h) + _blocks(h) * _blocks(o))
        return {"bytes": weights + 2 * h + t * e * (3 * h + n + h), "flops": 2 * t * (n * h + h * o)}
    rows, cols = case["rows"], case["cols"]
    values = rows * cols
    if kind == "norm":
        by = values * e * (3 if case["residual"] else 1) + cols * e
        by += rows * (cols + 4 * _blocks(cols)) if case["fp8"] else values * e
        return {"bytes": by, "flops": 6 * values}
    by = values * (e + 1) + 4 * _blocks(cols) * (rows if kind == "quant_x" else _blocks(rows))
    return {"bytes": by, "flops": 3 * values}


# ---------------------------------------------------------------- inputs

def _angles_per_token(case):
    """(angle of each pair per position, magnitude) of a case's scaling, on the host in 64 bits: plain powers of the
    base; all divided (linear); the base raised (ntk); slow pairs divided, fast ones kept and a ramp between them over
    the turns that a pair makes in the original length (yarn, smooth)."""
    rot, how = case["rot"], case["scaling"]
    base, factor, length = 10000.0, 8.0, 8192.0
    if how == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if how == "linear":
        return [x / factor for x in f], 1.0
    if how == "yarn":
        def pair(turns):
            return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    if how == "smooth":
        keep = [min(max((length * x / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0) for x in f]
        return [x * r + x / factor * (1 - r) for x, r in zip(f, keep)], 1.0
    return f, 1.0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)


def _quantize(x, rows_too):
    """x float32 [R, C] -> e4m3 codes and scales of 1 x 128 groups or 128 x 128 blocks: the largest magnitude goes to
    448. Quotients of short values lie on the border between two codes now and then: they are taken in 64 bits."""
    rows, cols = x.shape
    g = _GROUP if rows_too else 1
    pad = torch.nn.functional.pad(x, (0, -cols % _GROUP, 0, -rows % g))
    b = pad.unflatten(0, (-1, g)).unflatten(2, (-1, _GROUP))
    amax = b.abs().amax((1, 3), keepdim=True).clamp(min=2.0 ** -100)
    codes = (b.double() * 448 / amax.double()).flatten(2).flatten(0, 1)[:rows, :cols]
    return codes.float().to(_E4M3).contiguous(), (amax / torch.full_like(amax, 448.0))[:, 0, :, 0].contiguous()


def _activations(rows, cols, gen):
    """Unit values with a few large channels."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x[:, torch.randint(cols, (3,), generator=gen, device="cuda")] *= 8.0
    return x


def _weights(n, k, gen):
    """e4m3 weights of unit gain, rows of different size."""
    w = torch.randn(n, k, generator=gen, device="cuda") * (k ** -0.5)
    return _quantize(w * (0.5 + torch.rand(n, 1, generator=gen, device="cuda")), True)


def prepare(case, seed):
    gen = _gen(seed)
    dt = _DT[case["dtype"]]
    kind = case["kind"]
    st = {"case": case, "eps": 1e-6}
    if kind in ("rope", "layer"):
        # what a plan gives: each row's position in its request
        t = case["tokens"]
        st["positions"] = torch.randint(case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        f, st["mscale"] = _angles_per_token(case)
        st["inv_freq"] = torch.tensor(f, dtype=torch.float64).cuda()
        if kind == "rope":
            # rows as slices of one projection's output
            qkv = torch.randn(t, case["hq"] + 2 * case["hkv"], case["d"], generator=gen, device="cuda").to(dt)
            st["q"], st["k"], _ = qkv.split([case["hq"], case["hkv"], case["hkv"]], 1)
            return st
        h, o = case["hidden"], case["hq"] * case["d"]
        st["x"], st["residual"] = _activations(t, h, gen).to(dt), _activations(t, h, gen).to(dt)
        st["gain"] = (1 + 0.1 * torch.randn(h, generator=gen, device="cuda")).to(dt)
        st["w_qkv"] = _weights(o + 2 * case["hkv"] * case["d"], h, gen)
        st["w_out"] = _weights(h, o, gen)
        return st
    if kind == "mm":
        st["x"] = _quantize(_activations(case["m"], case["k"], gen), False)
        st["w"] = _weights(case["n"], case["k"], gen)
        return st
    rows, cols = case["rows"], case["cols"]
    if kind == "quant_w":
        st["w"] = (torch.randn(rows, cols, generator=gen, device="cuda") * 0.02).to(dt)
        return st
    st["x"] = _activations(rows, cols, gen).to(dt)
    if kind == "norm":
        st["residual"] = _activations(rows, cols, gen).to(dt) if case["residual"] else None
        st["gain"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(dt)
    return st


# ---------------------------------------------------------------- plain forms

def _rope(st, q, k):
    rot = st["case"]["rot"]
    a = st["positions"].double()[:, None] * st["inv_freq"]      # (far angles need 64 bits)
    cos, sin = (f(a).mul_(st["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))
    return [_turned(x, cos, sin, rot, st["case"]["interleaved"]) for x in (q, k)]


def _turned(x, cos, sin, rot, interleaved):
    r = x[..., :rot].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y.to(x.dtype), x[..., rot:]], -1)


def _norm(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + st["eps"]) * st["gain"].float()
    return h.to(st["x"].dtype), y


def _values(codes, scales):
    """What e4m3 codes with scales of 1 x 128 groups or 128 x 128 blocks stand for, float32."""
    rows, cols = codes.shape
    s = scales.repeat_interleave(_GROUP, 1)[:, :cols]
    if scales.shape[0] != rows:
        s = s.repeat_interleave(_GROUP, 0)[:rows]
    return codes.float() * s


def _mm(w, x, dt):
    return (_values(*x) @ _values(*w).t()).to(dt)


def run(st):
    c = st["case"]
    kind = c["kind"]
    dt = _DT[c["dtype"]]
    if own:
        return _run_own(st, dt)
    if kind == "rope":
        return _rope(st, st["q"], st["k"])
    if kind == "quant_x":
        return _quantize(st["x"].float(), False)
    if kind == "quant_w":
        return _quantize(st["w"].float(), True)
    if kind == "mm":
        return _mm(st["w"], st["x"], dt)
    h, y = _norm(st)
    if kind == "norm":
        out = {"codes_scales": _quantize(y, False)} if c["fp8"] else {"out": y.to(dt)}
        return {"residual": h, **out} if c["residual"] else out
    qkv = _mm(st["w_qkv"], _quantize(y, False), dt).unflatten(1, (-1, c["d"]))
    q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
    q, k = _rope(st, q, k)
    # (the attention between them is measured elsewhere; the rotated queries stand for its outputs)
    return {"residual": h, "q": q, "k": k, "v": v, "out": _mm(st["w_out"], _quantize(q.flatten(1).float(), False), dt)}


def _run_own(st, dt):
    import gemm_affine_int4_gb300 as g4
    c = st["case"]
    kind = c["kind"]
    if kind == "rope":
        return list(g4.gai4_rope(st["q"], st["k"], st["positions"], st["inv_freq"], interleaved=c["interleaved"],
                                 mscale=st["mscale"]))
    if kind == "quant_x":
        return g4.gai4_quantize_x_fp8(st["x"])
    if kind == "quant_w":
        return g4.gai4_quantize_fp8(st["w"])
    if kind == "mm":
        return g4.gai4_fp8_mm_t(*st["w"], *st["x"], dtype=dt)
    n = g4.gai4_rms_norm(st["x"], st["gain"], eps=st["eps"], residual=st["residual"],
                         fp8=kind == "layer" or c["fp8"])
    if kind == "norm":
        out = {"codes_scales": (n.codes, n.scales)} if c["fp8"] else {"out": n.out}
        return {"residual": n.residual, **out} if c["residual"] else out
    qkv = g4.gai4_fp8_mm_t(*st["w_qkv"], n.codes, n.scales, dtype=dt).unflatten(1, (-1, c["d"]))
    q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
    g4.gai4_rope(q, k, st["positions"], st["inv_freq"], interleaved=c["interleaved"], mscale=st["mscale"], q_out=q,
                 k_out=k)
    x = g4.gai4_quantize_x_fp8(q.flatten(1))
    return {"residual": n.residual, "q": q, "k": k, "v": v, "out": g4.gai4_fp8_mm_t(*st["w_out"], *x, dtype=dt)}


# ---------------------------------------------------------------- values in 64 bits

def _nearest_e4m3(v):
    """The e4m3 value nearest to v, |v| <= 448 (ties to even), in float64: three bits after the leading one, steps of
    2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantize(x, rows_too):
    rows, cols = x.shape
    codes = torch.empty_like(x)
    g = _GROUP if rows_too else rows
    scales = torch.empty(_blocks(rows) if rows_too else rows, _blocks(cols), dtype=torch.float64, device=x.device)
    for i in range(0, rows, g):
        for j in range(0, cols, _GROUP):
            part = x[i:i + g, j:j + _GROUP]
            s = part.abs().amax() if rows_too else part.abs().amax(1, keepdim=True)
            s = s.clamp(min=2.0 ** -100)
            codes[i:i + g, j:j + _GROUP] = _nearest_e4m3(part * 448 / s)
            scales[i // g if rows_too else slice(None), j // _GROUP] = s / 448 if rows_too else s[:, 0] / 448
    return codes, scales


def _exact_rope(st, x):
    c = st["case"]
    rot = c["rot"]
    a = torch.outer(st["positions"].double(), st["inv_freq"])
    turn = torch.polar(torch.full_like(a, st["mscale"]), a)[:, None]
    y = x.double().clone()
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_norm(st):
    h = st["x"].double()
    if st["residual"] is not None:
        h = h + st["residual"].double()
    return h, h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + st["eps"]) * st["gain"].double()


def _exact_mm(w, x):
    (wc, ws), (xc, xs) = w, x
    n, k = wc.shape
    out = torch.zeros(xc.shape[0], n, dtype=torch.float64, device=wc.device)
    for j in range(_blocks(k)):
        at = slice(j * _GROUP, (j + 1) * _GROUP)
        part = wc[:, at].double() * ws[:, j].double().repeat_interleave(_GROUP)[:n, None]
        out.addmm_(xc[:, at].double() * xs[:, j].double()[:, None], part.t())
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return [_exact_rope(st, x) for x in (st["q"], st["k"])]
    if kind == "quant_x":
        return _exact_quantize(st["x"].double(), False)
    if kind == "quant_w":
        return _exact_quantize(st["w"].double(), True)
    if kind == "mm":
        return _exact_mm(st["w"], st["x"])
    h, y = _exact_norm(st)
    if kind == "norm":
        out = {"codes_scales": _exact_quantize(y, False)} if case["fp8"] else {"out": y}
        return {"residual": h, **out} if case["residual"] else out
    # each operator takes the rows that the one before it has rounded to the case's type
    dt = _DT[case["dtype"]]
    qkv = _exact_mm(st["w_qkv"], _exact_quantize(y, False)).unflatten(1, (-1, case["d"]))
    v = qkv[:, case["hq"] + case["hkv"]:]
    q, k, _ = qkv.to(dt).split([case["hq"], case["hkv"], case["hkv"]], 1)
    q, k = _exact_rope(st, q), _exact_rope(st, k)
    x = _exact_quantize(q.to(dt).double().flatten(1), False)
    return {"residual": h, "q": q, "k": k, "v": v, "out": _exact_mm(st["w_out"], x)}
