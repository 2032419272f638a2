"""Plain 64-bit implementation of the paged 4-bit key/value cache operators, and the error bounds of their tests.

Error bounds of the attention outputs (u = unit roundoff of T, f = 2^-24; A = sum_j p_j (|s c_j| + |b|) and B =
sum_j p_j |v_j| of the output element, S = scale * sum_d |q_d| (|s c_d| + |b|) the largest over the keys):
  few rows, bf16 / f16: the codes are exact; probabilities times value scales are rounded to binary16 (2^-11, and a
    quantum of 2^-38 of the largest). Scores carry binary32 sums of a head's 128 products and two roundings per group:
    140 f S each; the exponential's argument and result another 2^-21 (1 + S). So A (2^-11 + 2 * (140 f S + 2^-21 (1 + S))
    + n f), n keys summed in binary32.
  few rows, f32: the same with probabilities split in two binary16 parts (2^-21) and queries in two (2^-21 S).
  many rows: keys, values and probabilities are rounded once to T (u each): 2 u S + B (...) as above with 2 u for value
    and probability.
and one spacing of T for the rounded output.
"""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}
TINY = {"bf16": 2.0**-133, "f16": 2.0**-24, "f32": 2.0**-149}


def quantize64(x, gs, dt):
    """x [..., D] tensor of type dt -> codes int64 [..., D], scales and biases in dt (binary32 steps by numpy)."""
    f = x.float().cpu().numpy()
    g = f.reshape(f.shape[:-1] + (-1, gs))
    lo, hi = g.min(-1), g.max(-1)
    s = torch.from_numpy((hi - lo) / np.float32(15)).to(dt)
    b = torch.from_numpy(lo).to(dt)
    sf, bf = s.float().numpy()[..., None], b.float().numpy()[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.rint((g - bf) / sf), 0, 15)
    q = np.where(sf == 0, 0, q)
    return torch.from_numpy(q.reshape(f.shape)).long(), s, b


def pack(codes):
    w = (codes.reshape(codes.shape[:-1] + (-1, 8)) << torch.arange(0, 32, 4)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def unpack(w):
    return ((w.long().unsqueeze(-1) >> torch.arange(0, 32, 4, device=w.device)) & 15).flatten(-2)


def random_cache(nb, hkv, page, d, gs, dt, seed, spread=1.0, device="cuda"):
    """A pool of quantized normal rows with a wide spread of scales."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(nb, hkv, page, d, generator=g)
    x = x * torch.exp(spread * torch.randn(nb, hkv, page, 1, generator=g)) + 0.3 * torch.randn(hkv, 1, d, generator=g)
    codes, s, b = quantize64(x.to(DT[dt]), gs, DT[dt])
    return tuple(t.to(device) for t in (pack(codes), s, b))


def rows64(cache, pages, offs, gs):
    """(values, |s c| + |b|) of rows, float64 [rows, hkv, d]."""
    w, s, b = cache
    c = unpack(w[pages, :, offs]).double()
    s = s[pages, :, offs].double().repeat_interleave(gs, -1)
    b = b[pages, :, offs].double().repeat_interleave(gs, -1)
    return s * c + b, (s * c).abs() + b.abs()


def attention64(q, k_cache, v_cache, table, kv_lens, cu_q, gs, scale, window, dt, many_rows=False):
    """(out, bound, lse, lse_bound) in float64."""
    nb, hkv, page = k_cache[0].shape[:3]
    n, hq, d = q.shape
    g = hq // hkv
    u, f = U[dt], 2.0**-24
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((n, hq), -np.inf, dtype=torch.float64, device=q.device)
    lse_bound = torch.zeros_like(lse)
    for r in range(len(kv_lens)):
        a, e, kv = cu_q[r], cu_q[r + 1], min(kv_lens[r], table.shape[1] * page)
        if a == e or kv <= 0:
            continue
        j = torch.arange(kv, device=q.device)
        blocks = table[r, j // page].long()
        there = (blocks >= 0) & (blocks < nb)
        blocks = torch.where(there, blocks, 0)
        (k, ka), (v, va) = (rows64(c, blocks, j % page, gs) for c in (k_cache, v_cache))
        pos = (kv - (e - a) + torch.arange(e - a, device=q.device))[:, None]
        see = (j <= pos) & there
        if window:
            see &= j > pos - window
        any_ = see.any(1)
        # rows that no query sees may hold anything
        seen = see.any(0)
        k, ka, v, va = (torch.where(seen[:, None, None], t, 0.0) for t in (k, ka, v, va))
        for h in range(hkv):
            qh = q[a:e, h * g:(h + 1) * g].double()
            s = scale * torch.einsum("tgd,kd->tgk", qh, k[:, h])
            s = torch.where(see[:, None], s, -np.inf)
            S = abs(scale) * torch.einsum("tgd,kd->tgk", qh.abs(), ka[:, h])
            S = torch.where(see[:, None], S, 0.0).amax(-1)
            p = torch.softmax(s, -1).nan_to_num(0.0)
            out[a:e, h * g:(h + 1) * g] = p @ v[:, h]
            delta = 140 * f * S + 2.0**-21 * (1 + S) + (2.0**-21 * S if dt == "f32" else 0.0)
            sums = kv * f
            if many_rows and dt != "f32":
                delta = delta + u * S
                rel = (torch.exp(2 * delta) - 1) + 2 * u + sums
                bnd = rel[..., None] * (p @ v[:, h].abs())
            else:
                rel = (torch.exp(2 * delta) - 1) + (2.0**-21 if dt == "f32" else 2.0**-11) + sums
                bnd = rel[..., None] * (p @ va[:, h])
            bound[a:e, h * g:(h + 1) * g] = bnd
            lse[a:e, h * g:(h + 1) * g] = torch.where(any_[:, None], torch.logsumexp(s, -1), -np.inf)
            lse_bound[a:e, h * g:(h + 1) * g] = delta + sums + 2.0**-22 * (1 + lse[a:e, h * g:(h + 1) * g].abs())
    # one spacing of T
    ulp = torch.maximum(out.abs() * 2 * u, torch.tensor(TINY[dt], dtype=torch.float64))
    return out, bound + ulp, lse, lse_bound


def plan_reference(kv_lens, q_lens, table, free, count, page, num_tokens):
    """The step's bookkeeping, request by request, on Python lists (table and free as lists, updated copies returned)."""
    table, free = [list(t) for t in table], list(free)
    B, width = len(kv_lens), len(table[0])
    pages = lambda n: -(-n // page)  # noqa: E731
    gave = sum(pages(l) for l, n in zip(kv_lens, q_lens) if n < 0)
    took = sum(pages(l + n) - pages(l) for l, n in zip(kv_lens, q_lens) if n >= 0)
    total = sum(max(n, 0) for n in q_lens)
    wrong = int(any(l < 0 for l in kv_lens) or count < 0 or count + gave > len(free))
    info = [0 if wrong else max(0, took - count - gave),
            sum(pages(l + max(n, 0)) > width for l, n in zip(kv_lens, q_lens)), max(0, total - num_tokens), wrong]
    if any(info):
        return dict(table=table, free=free, slots=[-1] * num_tokens, positions=[0] * num_tokens, cu_q=[0] * (B + 1),
                    kv_lens=list(kv_lens), count=count, info=info)
    stack = free[:count]
    for r in range(B):
        if q_lens[r] < 0:
            stack += table[r][:pages(kv_lens[r])]
    free[:len(stack)] = stack
    slots, positions, cu, new = [], [], [0], []
    for r in range(B):
        l, n = kv_lens[r], max(q_lens[r], 0)
        if q_lens[r] >= 0:
            for b in range(pages(l), pages(l + n)):
                table[r][b] = stack.pop()
            for j in range(l, l + n):
                slots.append(table[r][j // page] * page + j % page)
                positions.append(j)
        cu.append(cu[-1] + n)
        new.append(0 if q_lens[r] < 0 else l + n)
    pad = num_tokens - len(slots)
    return dict(table=table, free=free, slots=slots + [-1] * pad, positions=positions + [0] * pad, cu_q=cu,
                kv_lens=new, count=len(stack), info=info)
