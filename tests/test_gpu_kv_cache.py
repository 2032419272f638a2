"""Paged 4-bit key/value cache on the GPU: gai4_kv_plan, gai4_kv_append and gai4_kv_read against plain
implementations, exactly, and gai4_kv_attention against the 64-bit one within the bounds of kv_ref.py."""
import random

import numpy as np
import pytest
import torch

import gemm_affine_int4_gb300 as g4
from kv_ref import DT, attention64, pack, plan_reference, quantize64, random_cache

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan

def run_plan(kv, q, table, free, count, page, T, stream=None):
    tb, fr = i32(table), i32(free)
    p = g4.gai4_kv_plan(i32(kv), i32(q), tb, fr, i32([count]), page, T, stream=stream)
    torch.cuda.synchronize()
    got = dict(table=tb.tolist(), free=fr.tolist(), slots=p.slots.tolist(), positions=p.positions.tolist(),
               cu_q=p.cu_q.tolist(), kv_lens=p.kv_lens.tolist(), count=int(p.free_count), info=p.info.tolist())
    return got


def make_step(rng, B, page, width, q_hi, finished):
    kv = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, width * page)]) for _ in range(B)]
    kv = [min(k, width * page) for k in kv]
    q = [rng.choice([0, 1, rng.randint(0, q_hi)]) for _ in range(B)]
    q = [min(n, width * page - k) for n, k in zip(q, kv)]
    for i in range(finished):
        q[rng.randrange(B)] = -1
    need = sum(-(-(k + max(n, 0)) // page) for n, k in zip(q, kv))
    ids = list(range(need + 3))
    rng.shuffle(ids)
    table, at = [], 0
    for k in kv:
        m = -(-k // page)
        table.append(ids[at:at + m] + [-1] * (width - m))
        at += m
    free = ids[at:]
    count = len(free)
    free = free + [-7] * (at + 2)      # room for what finished requests give back
    return kv, q, table, free, count


@pytest.mark.parametrize("B,page,width,q_hi,finished", [
    (1, 16, 4, 0, 0), (1, 64, 8, 500, 0), (1, 16, 3, 0, 1), (2, 256, 2, 3, 1), (31, 16, 9, 40, 3), (33, 32, 5, 1, 0),
    (64, 64, 40, 1, 0), (200, 128, 6, 300, 150), (1000, 16, 12, 60, 90), (1025, 32, 4, 5, 4), (2500, 16, 2, 2, 100),
    (8192, 16, 2, 1, 13)])
def test_plan(B, page, width, q_hi, finished):
    rng = random.Random(B * 31 + page)
    step = make_step(rng, B, page, width, q_hi, finished)
    T = sum(max(n, 0) for n in step[1])
    for pad in (0, 37):
        want = plan_reference(*step, page, T + pad)
        assert want["info"] == [0, 0, 0, 0]
        assert run_plan(*step, page, T + pad) == want


def test_plan_no_new_tokens():
    assert run_plan([0, 5], [0, 0], [[-1], [3]], [9], 1, 16, 0)["cu_q"] == [0, 0, 0]


def test_plan_reuses_pages_freed_in_the_same_step():
    # nothing free at first: request 1's pages feed requests 0 and 2
    args = ([32, 40, 0], [1, -1, 17], [[5, -1], [7, 2], [-1, -1]], [0] * 8, 0, 32, 18)
    got = run_plan(*args)
    assert got == plan_reference(*args)
    assert got["table"] == [[5, 2], [7, 2], [7, -1]] and got["count"] == 0


@pytest.mark.parametrize("change,info", [
    (dict(count=2), [2, 0, 0, 0]),                 # 4 pages needed, 2 there
    (dict(q=[1, 20, 100], width=3), None),         # a row of the table too short
    (dict(T=2), [0, 0, 48, 0]),                    # more new tokens than rows
    (dict(kv=[-1, 10, 0]), None),                  # negative length
    (dict(count=-1), [0, 0, 0, 1]),
    (dict(q=[1, -1, 3], count=7), None),           # the freed page does not fit the list
])
def test_plan_refuses_a_step_as_a_whole(change, info):
    a = dict(kv=[16, 10, 0], q=[1, 20, 29], width=4, count=7, T=60)
    a.update(change)
    table = [[1] + [-1] * (a["width"] - 1), [2] + [-1] * (a["width"] - 1), [-1] * a["width"]]
    args = (a["kv"], a["q"], table, [10, 11, 12, 13, 14, 15, 16], a["count"], 16, a["T"])
    want = plan_reference(*args)
    got = run_plan(*args)
    assert any(want["info"]) and got == want
    if info is not None:
        assert got["info"] == info


# ------------------------------------------------------------------ append, read

def put(x, slots, page, nb, gs, dt, canary=None):
    """Expected (packed, scales, biases) after rows x [T, H, D] went to their slots of a zero cache."""
    T, H, D = x.shape
    codes, s, b = quantize64(x, gs, DT[dt])
    w = torch.zeros(nb, H, page, D // 8, dtype=torch.int32)
    sc, bi = torch.zeros(nb, H, page, D // gs, dtype=DT[dt]), torch.zeros(nb, H, page, D // gs, dtype=DT[dt])
    for i, t in enumerate(slots):
        if 0 <= t < nb * page:
            w[t // page, :, t % page], sc[t // page, :, t % page], bi[t // page, :, t % page] = pack(codes[i]), s[i], b[i]
    return w, sc, bi


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,D,gs,page", [(1, 1, 64, 32, 16), (1, 8, 128, 64, 64), (7, 3, 64, 64, 32),
                                           (65, 2, 128, 32, 16), (130, 5, 128, 128, 256), (33, 1, 128, 64, 128)])
def test_append_and_read(dt, T, H, D, gs, page):
    nb = -(-T // page) + 3
    g = torch.Generator().manual_seed(T + H + D + gs)
    k, v = (torch.randn(T, H, D, generator=g) * torch.exp(2 * torch.randn(T, H, 1, generator=g)) for _ in range(2))
    k[0, 0, :gs] = 1.25          # a constant group: scale 0
    v[-1, -1] = 0.0
    k, v = k.to(DT[dt]), v.to(DT[dt])
    slots = torch.randperm(nb * page, generator=g)[:T].tolist()
    if T > 3:
        slots[1], slots[3] = -1, nb * page       # outside the pool: skipped
    kc, vc = (g4.gai4_kv_cache(nb, H, page, D, gs, DT[dt]) for _ in range(2))
    st = torch.tensor(slots, dtype=torch.int64, device="cuda")
    g4.gai4_kv_append(k.cuda(), v.cuda(), st, kc, vc, group_size=gs)
    for x, c in ((k, kc), (v, vc)):
        for got, want in zip(c, put(x, slots, page, nb, gs, dt)):
            assert torch.equal(got.cpu(), want)
        # the rows as gai4_quantize and gai4_dequantize have them
        rows = x.float().reshape(T * H, D).cuda()
        wq, s, b = g4.gai4_quantize(rows, 4, gs, DT[dt])
        val = g4.gai4_dequantize(wq, s, b, 4, gs).view(T, H, D)
        val[[i for i, t in enumerate(slots) if not 0 <= t < nb * page]] = 0.0
        assert torch.equal(g4.gai4_kv_read(c, st, group_size=gs), val)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (1, 0), (0, 1), (5, 3)])
def test_append_strided_rows(dt, pad, off):
    T, H, D, gs, page, nb = 21, 2, 64, 32, 16, 4
    g = torch.Generator().manual_seed(5)
    base = torch.randn(T * (H * D + pad) + off, generator=g).to(DT[dt])
    k = torch.as_strided(base, (T, H, D), (H * D + pad, D, 1), off)
    v = torch.randn(T, 3 * H, D, generator=g).to(DT[dt])[:, H:2 * H]
    slots = torch.randperm(nb * page, generator=g)[:T]
    kc, vc = (g4.gai4_kv_cache(nb, H, page, D, gs, DT[dt]) for _ in range(2))
    kg = torch.as_strided(base.cuda(), k.shape, k.stride(), off)
    vg = torch.randn(T, 3 * H, D).to(DT[dt]).cuda()
    vg[:, H:2 * H] = v.cuda()
    g4.gai4_kv_append(kg, vg[:, H:2 * H], slots.cuda(), kc, vc, group_size=gs)
    for x, c in ((k, kc), (v, vc)):
        for got, want in zip(c, put(x, slots.tolist(), page, nb, gs, dt)):
            assert torch.equal(got.cpu(), want)


def test_append_codes_at_rounding_ties():
    """Quotients at and around every half: the codes are those of an IEEE division."""
    for dt in ("bf16", "f16", "f32"):
        D, gs, T = 64, 64, 400
        g = torch.Generator().manual_seed(11)
        x = torch.rand(T, 1, D, generator=g)
        x[:, :, 0], x[:, :, 1] = 0.0, 15.0
        x[:, :, 2:] = (torch.randint(0, 30, (T, 1, D - 2), generator=g) / 2) + \
            torch.randint(-2, 3, (T, 1, D - 2), generator=g) * 2.0**-21
        x = (x * torch.exp(torch.randn(T, 1, 1, generator=g))).to(DT[dt])
        kc, vc = (g4.gai4_kv_cache(-(-T // 16), 1, 16, D, gs, DT[dt]) for _ in range(2))
        slots = torch.arange(T)
        g4.gai4_kv_append(x.cuda(), x.cuda(), slots.cuda(), kc, vc, group_size=gs)
        for got, want in zip(kc, put(x, slots.tolist(), 16, -(-T // 16), gs, dt)):
            assert torch.equal(got.cpu(), want)


def test_append_writes_only_its_rows():
    nb, H, page, D, gs = 3, 2, 16, 128, 64
    parts = []
    for _ in range(2):
        parts.append((torch.full((nb, H, page, D // 8), 0x5A5A5A5A, dtype=torch.int32, device="cuda"),
                      torch.full((nb, H, page, D // gs), 7.0, dtype=torch.bfloat16, device="cuda"),
                      torch.full((nb, H, page, D // gs), 7.0, dtype=torch.bfloat16, device="cuda")))
    k = torch.randn(2, H, D, device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([page + 3, -5], device="cuda")
    g4.gai4_kv_append(k, k, slots, *parts, group_size=gs)
    for c in parts:
        for t, old in zip(c, (0x5A5A5A5A, 7, 7)):
            same = (t == old).all(-1).cpu()
            same[1, :, 3] = True
            assert bool(same.all())


# ------------------------------------------------------------------ attention

def check(q, kc, vc, table, kv, cu, gs, dt, window=0, scale=None, max_q=None, many=False, pad_rows=0, **kw):
    n, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    if max_q is None:
        max_q = max(b - a for a, b in zip(cu, cu[1:]))
    lse = torch.full((n, hq), 5.0, device="cuda")
    out = torch.full((n, hq, d), float("nan"), dtype=DT[dt], device="cuda")
    got = g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=gs, scale=scale, window=window,
                               max_q_len=max_q, out=out, lse=lse, **kw)
    assert got is out and g4.gai4_last_device_status() == 0
    ref, bound, rl, lb = attention64(q, kc, vc, table, kv, cu, gs, scale, window, dt, many)
    err = (out.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} outside; worst {float((err / bound).nan_to_num(1e30).max()):.3g} at "
        f"{np.unravel_index(int((err / bound).nan_to_num(1e30).argmax()), err.shape)}")
    empty = rl == -np.inf
    assert torch.equal(lse == -np.inf, empty)
    le = torch.where(empty, 0.0, (lse.double() - rl).abs())
    assert bool((le <= lb).all()), f"lse: worst {float(le.max()):.3g}"
    return out


def problem(kv, q_lens, hkv, g, d, gs, page, dt, seed, spare=3, width_extra=1):
    """Queries, caches and a table whose pages are in random order; every slot that no request owns holds NaN scales
    and biases, and every table entry past a request's pages is invalid."""
    gen = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-k // page) for k in kv)) + width_extra
    nb = sum(-(-k // page) for k in kv) + spare
    perm = torch.randperm(nb, generator=gen).tolist()
    table = torch.full((len(kv), width), -1, dtype=torch.int32)
    used = torch.zeros(nb, page, dtype=torch.bool)
    at = 0
    for r, k in enumerate(kv):
        for b in range(-(-k // page)):
            table[r, b] = perm[at]
            used[perm[at], :min(page, k - b * page)] = True
            at += 1
    table[:, -1] = torch.where(table[:, -1] < 0, nb + 5, table[:, -1])
    kc, vc = (list(random_cache(nb, hkv, page, d, gs, dt, seed + i, 0.5)) for i in range(2))
    hide = ~used.cuda()[:, None, :, None]
    for c in (kc, vc):
        c[1] = c[1].masked_fill(hide, float("nan"))
        c[2] = c[2].masked_fill(hide, float("inf"))
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], hkv * g, d, generator=gen).to(DT[dt]).cuda()
    return q, tuple(kc), tuple(vc), table.cuda(), list(kv), cu


LAYOUTS = [(1, 1, 64, 32, 16), (2, 4, 64, 64, 32), (8, 4, 128, 64, 64), (1, 8, 128, 32, 16), (3, 7, 128, 128, 128),
           (1, 16, 128, 64, 256), (2, 5, 64, 32, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hkv,g,d,gs,page", LAYOUTS)
def test_one_token(dt, hkv, g, d, gs, page):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1000]
    check(*problem(kv, [1] * len(kv), hkv, g, d, gs, page, dt, 17), gs, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kv", [[1], [37], [700], [9000], [40000, 3], [2049, 1, 8191]])
def test_one_token_lengths(dt, kv):
    check(*problem(kv, [1] * len(kv), 2, 4, 128, 64, 64, dt, 23), 64, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_no_keys_no_queries(dt):
    """Requests without cached tokens, without queries, and with more queries than tokens: rows that see nothing."""
    kv, q = [0, 5, 3, 0, 70, 1], [1, 0, 5, 2, 1, 4]
    a = problem(kv, q, 2, 3, 64, 32, 16, dt, 3)
    out = check(*a, 32, dt)
    assert bool((out[:1] == 0).all()) and bool((out[1:3] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_after_the_last_request(dt):
    q, kc, vc, table, kv, cu = problem([100, 30], [1, 2], 2, 4, 128, 64, 32, dt, 9)
    q = torch.cat([q, torch.full((5,) + q.shape[1:], float("nan"), dtype=q.dtype, device="cuda")])
    out = check(q, kc, vc, table, kv, cu, 64, dt)
    assert bool((out[3:] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("q_len", [1, 3])
def test_window(dt, window, q_len):
    kv = [3, 16, 99, 100, 101, 640, 1500]
    check(*problem(kv, [q_len] * len(kv), 2, 4, 128, 64, 32, dt, 31), 64, dt, window=window)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width_extra,window", [(0, 0), (1, 0), (60, 300), (60, 510), (60, 511)])
@pytest.mark.parametrize("q_len", [1, 2])
def test_units_up_to_and_above_512_tokens(dt, width_extra, window, q_len):
    """Block tables of 512 tokens and of one page more; windows that with the queries end at or above 512."""
    kv = [512, 511, 449, 448, 65, 64, 1, 0, 130, 512, 20]
    q = [min(q_len, k) for k in kv]
    check(*problem(kv, q, 2, 4, 128, 64, 16, dt, 47, width_extra=width_extra), 64, dt, window=window)


def test_largest_query_length_is_only_a_hint():
    """max_q_len picks the kernel: any value gives the rows their answer, within the wider bound."""
    a = problem([70, 300, 5], [1, 40, 3], 2, 4, 64, 32, 32, "bf16", 49)
    for max_q in (0, 1, 2, 3, 8, 9, 40, 1000, 2**62):
        check(*a, 32, "bf16", max_q=max_q, many=True)


def test_window_pages_may_be_gone():
    """Pages that the window has passed: invalid table entries in their place."""
    q, kc, vc, table, kv, cu = problem([700], [2], 2, 4, 128, 64, 32, "f16", 37)
    table = table.clone()
    table[0, :15] = -1            # window of 200 starts at 499, page 15
    check(q, kc, vc, table, kv, cu, 64, "f16", window=200)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hkv,g,d,gs,page", LAYOUTS)
def test_few_tokens(dt, hkv, g, d, gs, page):
    kv, q = [9, 70, 128, 200, 650], [3, 2, 4, 1, 4]
    check(*problem(kv, q, hkv, g, d, gs, page, dt, 41), gs, dt, many=4 * g > 32)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hkv,g,d,gs,page", LAYOUTS)
def test_chunks(dt, hkv, g, d, gs, page):
    """Many query rows per request, ragged, with and without older tokens."""
    kv, q = [150, 333, 40, 500, 7], [150, 77, 33, 1, 0]
    check(*problem(kv, q, hkv, g, d, gs, page, dt, 43), gs, dt, many=True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("window", [0, 1, 64, 200])
def test_chunk_lengths(dt, window):
    for kv, q in (([1], [1]), ([129], [129]), ([700], [300]), ([1025], [513]), ([5000], [130]), ([33, 2000], [40, 256])):
        check(*problem(kv, q, 2, 2, 128, 64, 64, dt, 47), 64, dt, many=True, window=window, max_q=4096)


def test_chunk_rows_that_see_nothing():
    kv, q = [0, 5, 100], [70, 90, 130]
    check(*problem(kv, q, 2, 4, 64, 32, 16, "bf16", 53), 32, "bf16", many=True)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_sharp_and_wide_values(dt, many):
    """Large scores (one key takes almost everything), value scales over many orders of magnitude, zero scales."""
    kv, q = [300, 17, 129], ([40] * 3 if many else [1] * 3)
    qq, kc, vc, table, kv, cu = problem([max(a, b) for a, b in zip(kv, q)], q, 2, 4, 128, 64, 32, dt, 59)
    g = torch.Generator(device="cuda").manual_seed(3)
    e = torch.randint(-9, 10 if dt == "bf16" else 3, vc[1].shape, generator=g, device="cuda")
    vc = (vc[0], (vc[1].float() * torch.exp2(e.float())).to(DT[dt]), (vc[2].float() * torch.exp2(e.float())).to(DT[dt]))
    vc[1][0], kc[1][1] = 0.0, 0.0
    check(qq * 8, kc, vc, table, kv, cu, 64, dt, many=many)
    check(qq, kc, vc, table, kv, cu, 64, dt, many=many, scale=0.0)
    check(qq, kc, vc, table, kv, cu, 64, dt, many=many, scale=-0.7)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("dt,kv,q,window,many", [
    ("bf16", 300, 1, 50, False), ("f16", 300, 3, 0, False), ("f16", 1000, 5, 70, False), ("f32", 300, 4, 0, False),
    ("f32", 500, 40, 100, False), ("bf16", 300, 100, 0, True), ("f16", 1100, 300, 130, True),
    ("bf16", 9000, 20, 5000, True)])
def test_rows_do_not_meet_tokens_they_do_not_see(dt, kv, q, window, many, what, value):
    """Scales or biases of one group that are not finite, at tokens that some rows see and others do not (and one that
    none sees): keys touch the rows that see them (an infinite score may be minus infinity), values the group's channels
    of these rows, and nothing else."""
    hkv, g, d, gs, page = 2, 4, 64, 32, 32
    qs, kc, vc, table, kvs, cu = problem([kv], [q], hkv, g, d, gs, page, dt, 53)
    clean, bound, _, _ = attention64(qs, kc, vc, table, kvs, cu, gs, d ** -0.5, window, dt, many)
    tokens = {kv - 1: 1, kv - 1 - q // 2: 2}                 # token: scale (1) or bias (2)
    if window:
        tokens.update({kv - q - window: 1, kv - q + 1 - window + q // 2: 2})
    cache = tuple(x.clone() for x in (kc if what == "k" else vc))
    for t, field in tokens.items():
        cache[field][int(table[0, t // page]), 1, t % page, 1] = value
    args = (qs, cache, vc) if what == "k" else (qs, kc, cache)
    out = g4.gai4_kv_attention(*args, table, i32(kvs), i32(cu), group_size=gs, scale=d ** -0.5, window=window, max_q_len=q)
    pos = torch.arange(kv - q, kv, device="cuda")
    hit = torch.zeros(q, dtype=torch.bool, device="cuda")
    for t in tokens:
        hit |= (t <= pos) & ((t > pos - window) if window else True)
    assert bool(hit.any()) and (q == 1 or not bool(hit.all()) or window)
    gone = torch.zeros(q, hkv * g, d, dtype=torch.bool, device="cuda")
    gone[hit, g:, 0 if what == "k" else gs:] = True
    if what == "v" or value != value:
        assert not bool(out[gone].isfinite().any())
    err = torch.where(gone, 0.0, (out.double() - clean).abs())
    assert bool((err <= bound).all()), f"{int((~(err <= bound)).sum())} outside"


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_extreme_queries(dt):
    """Query magnitudes from 2^-60 to 2^60 (scores stay finite through the scale), zero and tiny rows."""
    q, kc, vc, table, kv, cu = problem([130, 64, 9], [1, 1, 1], 1, 8, 64, 64, 16, dt, 61)
    for e, scale in ((-60, 2.0**57), (60, 2.0**-63), (-120, 2.0**117)):
        check((q.float() * 2.0**e).to(DT[dt]), kc, vc, table, kv, cu, 64, dt, scale=scale)
    check(torch.zeros_like(q), kc, vc, table, kv, cu, 64, dt)


@pytest.mark.parametrize("max_q", [1, 64])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 5)])
def test_strided_queries_and_outputs(pad, off, max_q):
    hkv, g, d, gs, dt = 2, 4, 128, 64, "bf16"
    q, kc, vc, table, kv, cu = problem([90, 700], [3, 30] if max_q > 1 else [1, 1], hkv, g, d, gs, 32, dt, 67)
    n, hq, _ = q.shape
    stride = hq * d + pad
    base = torch.full((n * stride + off,), float("nan"), dtype=q.dtype, device="cuda")
    qs = torch.as_strided(base, q.shape, (stride, d, 1), off)
    qs.copy_(q)
    many = max_q > 1
    want = check(q, kc, vc, table, kv, cu, gs, dt, many=many, max_q=max_q)
    raw = torch.full((n * stride + off + 64,), 3.0, dtype=q.dtype, device="cuda")
    out = torch.as_strided(raw, q.shape, (stride, d, 1), off)
    g4.gai4_kv_attention(qs, kc, vc, table, i32(kv), i32(cu), group_size=gs, max_q_len=max_q, out=out)
    assert torch.equal(out, want)
    rest = torch.ones_like(raw, dtype=torch.bool)
    torch.as_strided(rest, q.shape, (stride, d, 1), off).fill_(False)
    assert bool((raw[rest] == 3.0).all())


@pytest.mark.parametrize("dt,q_len", [("bf16", 1), ("f32", 2), ("f16", 100)])
def test_repeats_bit_for_bit_whatever_the_workspace_holds(dt, q_len):
    kv = [3000, 50, 128, 911]
    q, kc, vc, table, kv, cu = problem(kv, [min(q_len, k) for k in kv], 2, 4, 128, 64, 64, dt, 71)
    nbytes = g4.gai4_kv_attention_workspace_bytes(8, 2, 128, DT[dt])
    outs = []
    for fill in (0.0, float("nan"), -1e30):
        ws = torch.full((nbytes // 4 + 16,), fill, device="cuda")
        out = g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=64, max_q_len=q_len,
                                   workspace=ws[:nbytes // 4])
        assert bool((ws[nbytes // 4:].isnan() if fill != fill else ws[nbytes // 4:] == fill).all())
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_offsets_past_32_bits():
    """A pool of more than 2^31 words: the pages in use lie at its end."""
    hkv, d, gs, page, nb = 8, 128, 64, 256, 66000
    kv, cu, used = [300, 77], [0, 1, 2], 4
    small = random_cache(used, hkv, page, d, gs, "bf16", 5)
    big = (torch.zeros(nb, hkv, page, d // 8, dtype=torch.int32, device="cuda"),
           torch.zeros(nb, hkv, page, d // gs, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(nb, hkv, page, d // gs, dtype=torch.bfloat16, device="cuda"))
    assert big[0].numel() > 2**31
    for b, s in zip(big, small):
        b[-used:] = s
    table = torch.tensor([[nb - 2, nb - 4], [nb - 1, -1]], dtype=torch.int32, device="cuda")
    q = torch.randn(2, hkv * 4, d, device="cuda").bfloat16()
    check(q, big, big, table, kv, cu, gs, "bf16")
    check(q, big, big, table, kv, cu, gs, "bf16", max_q=64, many=True)
    k = torch.randn(3, hkv, d, device="cuda").bfloat16()
    slots = torch.tensor([nb * page - 1, nb * page - 300, 5], device="cuda")
    other = tuple(t.clone() for t in small)
    g4.gai4_kv_append(k, k, slots, big, big, group_size=gs)
    g4.gai4_kv_append(k[:2], k[:2], slots[:2] - (nb - used) * page, other, other, group_size=gs)
    for b, s in zip(big, other):
        assert torch.equal(b[-used:], s)
    assert torch.equal(g4.gai4_kv_read(big, slots[:2], group_size=gs),
                       g4.gai4_kv_read(other, slots[:2] - (nb - used) * page, group_size=gs))


def test_step_on_another_stream_and_in_a_graph():
    """plan, append and attention in sequence on a side stream, eagerly and captured: the same results."""
    hkv, g, d, gs, page, B = 2, 4, 128, 64, 32, 5
    kvl, ql = [0, 31, 64, 200, 10], [7, 1, 1, 3, 0]
    width, nb = 9, 40
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).tolist()
    table, at = [], 0
    for k in kvl:
        m = -(-k // page)
        table.append(perm[at:at + m] + [-1] * (width - m))
        at += m
    free = perm[at:]
    T = sum(ql)
    gen = torch.Generator(device="cuda").manual_seed(7)
    qkv = torch.randn(T, (g + 2) * hkv, d, generator=gen, device="cuda").bfloat16()
    q, k, v = qkv.split([g * hkv, hkv, hkv], 1)
    pools = [random_cache(nb, hkv, page, d, gs, "bf16", i) for i in (1, 2)]
    ws = torch.empty(g4.gai4_kv_attention_workspace_bytes(g * hkv, hkv, d, torch.bfloat16) // 4 + 4, device="cuda")
    results = []
    kv_t, q_t, count = i32(kvl), i32(ql), i32([len(free)])

    def step(tb, fr, kc, vc, out, plan=None):
        p = g4.gai4_kv_plan(kv_t, q_t, tb, fr, count, page, T, out=plan)
        g4.gai4_kv_append(k, v, p.slots, kc, vc, group_size=gs)
        g4.gai4_kv_attention(q, kc, vc, tb, p.kv_lens, p.cu_q, group_size=gs, max_q_len=7, out=out, workspace=ws)
        return p

    for captured in (False, True):
        tb, fr = i32(table), i32(free)
        kc, vc = (tuple(t.clone() for t in c) for c in pools)
        out = torch.zeros(T, g * hkv, d, dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            if captured:
                plan = g4.gai4_kv_plan(kv_t, q_t, i32(table), i32(free), count, page, T)
                s.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    step(tb, fr, kc, vc, out, plan)
                graph.replay()
                p = plan
            else:
                p = step(tb, fr, kc, vc, out)
        s.synchronize()
        want = plan_reference(kvl, ql, table, free, len(free), page, T)
        assert p.slots.tolist() == want["slots"] and tb.tolist() == want["table"]
        results.append([out, *kc, *vc, p.slots])
        ref, bound, _, _ = attention64(q, kc, vc, tb, want["kv_lens"], want["cu_q"], gs, d ** -0.5, 0, "bf16")
        assert bool(((out.double() - ref).abs() <= bound).all())
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """A workspace of the current stream would be handed out again there while the call on `stream` still runs."""
    q, kc, vc, table, kv, cu = problem([70, 1500], [1, 1], 2, 4, 64, 32, 32, "bf16", 81)
    want = g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=32)
    kvd, cud, slots = i32(kv), i32(cu), torch.arange(5, device="cuda")
    plan = [i32([3, 0]), i32([1, 1]), i32([[0], [-1]]), i32([1, 2]), i32([2])]
    torch.cuda.synchronize()
    s, seen, empty = torch.cuda.Stream(), [], torch.empty

    def watched(*a, **k):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **k)
    monkeypatch.setattr(torch, "empty", watched)
    out = g4.gai4_kv_attention(q, kc, vc, table, kvd, cud, group_size=32, stream=s)
    g4.gai4_kv_read(kc, slots, group_size=32, stream=s)
    g4.gai4_kv_plan(*plan, 32, 2, stream=s)
    monkeypatch.undo()
    s.synchronize()
    assert torch.equal(out, want)
    assert len(seen) == 5 and set(seen) == {s.cuda_stream}


def test_plan_writes_only_its_outputs():
    rng = random.Random(3)
    kv, q, table, free, count = make_step(rng, 37, 16, 9, 50, 4)
    T = sum(max(n, 0) for n in q) + 5
    want = plan_reference(kv, q, table, free, count, 16, T)
    pads, parts = [], []
    for n, dt in ((T, torch.int64), (T, torch.int32), (38, torch.int32), (37, torch.int32), (1, torch.int32), (4, torch.int32)):
        raw = torch.full((n + 64,), 0x5A5A5A5A, dtype=dt, device="cuda")
        pads.append((raw, n))
        parts.append(raw[32:32 + n])
    tb, fr = i32(table), i32(free)
    p = g4.gai4_kv_plan(i32(kv), i32(q), tb, fr, i32([count]), 16, T, out=g4.KvPlan(*parts))
    assert p.slots.tolist() == want["slots"] and p.positions.tolist() == want["positions"]
    assert p.cu_q.tolist() == want["cu_q"] and p.kv_lens.tolist() == want["kv_lens"] and int(p.free_count) == want["count"]
    assert tb.tolist() == want["table"] and fr.tolist() == want["free"]
    for raw, n in pads:
        assert bool((raw[:32] == 0x5A5A5A5A).all()) and bool((raw[32 + n:] == 0x5A5A5A5A).all())


def test_append_infinite_and_nan_rows_stay_their_own():
    H, D, gs, page = 2, 64, 32, 16
    x = torch.randn(6, H, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    bad = x.clone()
    bad[1, 0, 3], bad[2, 1, 40], bad[4, 0, 0] = float("nan"), float("inf"), -float("inf")
    slots = torch.arange(6, device="cuda")
    caches = []
    for y in (x, bad):
        kc, vc = (g4.gai4_kv_cache(1, H, page, D, gs) for _ in range(2))
        g4.gai4_kv_append(y.cuda(), y.cuda(), slots, kc, vc, group_size=gs)
        caches.append(g4.gai4_kv_read(kc, slots, group_size=gs))
    touched = torch.zeros(6, H, D // gs, dtype=torch.bool)
    touched[1, 0, 0] = touched[2, 1, 1] = touched[4, 0, 0] = True
    same = (caches[0] == caches[1]).view(6, H, D // gs, gs).all(-1).cpu()
    assert bool((same | touched).all())


@pytest.mark.parametrize("dt,most", [("f32", 1e-5), ("f16", 4e-4)])
@pytest.mark.parametrize("d,gs", [(64, 32), (128, 64), (128, 128)])
def test_long_contexts_keep_their_precision(dt, most, d, gs):
    """The norm of the error over that of the output, where thousands of values nearly cancel: f16 by the rounding of
    the output (2^-12 on average over sqrt 3, 2.1e-4 at most) and of the probabilities times centred codes (as much
    again by one and a half); f32 by binary32 sums of a few 2^-24 of the centred codes."""
    q, kc, vc, table, kv, cu = problem([30000, 9000], [1, 1], 2, 4, d, gs, 64, dt, 83)
    out = g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=gs)
    ref, _, _, _ = attention64(q, kc, vc, table, kv, cu, gs, d ** -0.5, 0, dt)
    assert float((out.double() - ref).norm() / ref.norm()) < most


def test_many_steps_in_sequence():
    """Thirty decoding steps without a synchronisation between them: every step's attention sees its own append."""
    hkv, g, d, gs, page, B = 2, 4, 64, 32, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = (g4.gai4_kv_cache(12, hkv, page, d, gs) for _ in range(2))
    lens, free, count = i32([0] * B), i32(list(range(12))), i32([12])
    table = i32([[-1] * 4] * B)
    q_lens, xs, outs = i32([1] * B), [], []
    for _ in range(30):
        x = torch.randn(B, (g + 2) * hkv, d, generator=gen, device="cuda").bfloat16()
        q, k, v = x.split([g * hkv, hkv, hkv], 1)
        p = g4.gai4_kv_plan(lens, q_lens, table, free, count, page, B)
        g4.gai4_kv_append(k, v, p.slots, kc, vc, group_size=gs)
        outs.append(g4.gai4_kv_attention(q, kc, vc, table, p.kv_lens, p.cu_q, group_size=gs))
        lens, count = p.kv_lens, p.free_count
        xs.append(x)
    for n in (1, 2, 7, 16, 17, 30):
        q = xs[n - 1][:, :g * hkv]
        ref, bound, _, _ = attention64(q, kc, vc, table, [n] * B, [0, 1, 2, 3], gs, d ** -0.5, 0, "bf16")
        assert bool(((outs[n - 1].double() - ref).abs() <= bound).all()), n
