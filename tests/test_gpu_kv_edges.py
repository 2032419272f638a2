"""Edges of the paged 4-bit key/value cache on the GPU, within the bounds of kv_ref.py unless a test says otherwise."""
import numpy as np
import pytest
import torch

import gemm_affine_int4_gb300 as g4
from kv_ref import DT, U, attention64, rows64
from test_gpu_kv_cache import i32, problem

pytestmark = pytest.mark.gpu


def attend(q, kc, vc, table, kv, cu, gs, max_q, window=0, scale=None):
    """(out, lse) over sentinels."""
    n, hq, d = q.shape
    lse = torch.full((n, hq), 5.0, device="cuda")
    out = torch.full((n, hq, d), 7.0, dtype=q.dtype, device="cuda")
    g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=gs, max_q_len=max_q, window=window, scale=scale,
                         out=out, lse=lse)
    assert g4.gai4_last_device_status() == 0
    return out, lse


def compare(out, lse, ref, gone):
    """NaN in the (row, head) pairs of `gone`, the reference's values within its bounds in the others."""
    want, bound, rl, lb = ref
    assert bool(out[gone].isnan().all()) and bool(lse[gone].isnan().all()), "a row that should be NaN is not"
    stay = ~gone
    err = (out.double() - want).abs()[stay]
    assert bool((err <= bound[stay]).all()), f"{int((~(err <= bound[stay])).sum())} outside"
    empty = rl == -np.inf
    assert torch.equal((lse == -np.inf)[stay], empty[stay])
    le = torch.where(empty, 0.0, (lse.double() - rl).abs())[stay]
    assert bool((le <= lb[stay]).all())


# few rows: units of up to 512 tokens (not cut) and longer ones; many rows: one request (every unit cut) and many (most
# units whole)
FORMS = [("bf16", [60], 1, 0), ("f16", [60, 1, 33], 1, 0), ("f32", [60, 400], 1, 0), ("bf16", [5000], 1, 0),
         ("f16", [9000, 40], 1, 0), ("f32", [5000, 2100], 1, 0), ("f16", [3000, 70], 4, 0), ("bf16", [700], 2, 100),
         ("f32", [300, 900], 30, 0), ("bf16", [5000], 40, 0), ("f16", [300, 90], 60, 0), ("bf16", [70] * 170, 40, 0),
         ("f16", [150] * 160, 33, 50)]


@pytest.mark.parametrize("dt,kv,q_len,window", FORMS)
def test_nan_queries_give_nan_rows(dt, kv, q_len, window):
    q, kc, vc, table, kv, cu = problem(kv, [min(q_len, k) for k in kv], 2, 4, 64, 32, 32, dt, 91)
    many = q_len * 4 > 32
    gone = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    gone[0, 1] = gone[-1, 6] = gone[q.shape[0] // 2, 3] = True
    q[gone, 5] = float("nan")
    ref = attention64(torch.where(gone[:, :, None], 0.0, q), kc, vc, table, kv, cu, 32, 64 ** -0.5, window, dt, many)
    compare(*attend(q, kc, vc, table, kv, cu, 32, q_len, window), ref, gone)


def test_nan_queries_that_see_nothing_give_zeros():
    for q_len in (1, 40):
        q, kc, vc, table, kv, cu = problem([0, 5], [q_len] * 2, 2, 4, 64, 32, 32, "bf16", 92)
        q[0] = float("nan")
        out, lse = attend(q, kc, vc, table, kv, cu, 32, q_len)
        assert bool((out[0] == 0).all()) and bool((lse[0] == -np.inf).all())


@pytest.mark.parametrize("dt,kv,q_len,first,last", [
    ("bf16", 1, 1, 0, 1), ("f16", 1, 1, 0, 1), ("f32", 1, 1, 0, 1),          # the only key
    ("bf16", 33, 1, 32, 33), ("f16", 33, 2, 32, 33), ("f32", 65, 2, 64, 65),   # the newest, alone in its 32 tokens
    ("bf16", 400, 1, 0, 400), ("f16", 5000, 1, 0, 5000), ("f32", 5000, 2, 0, 5000),   # all
    ("bf16", 9000, 1, 3000, 6000), ("f32", 9000, 3, 4000, 7000),              # all that some blocks of a cut unit have
    ("bf16", 129, 40, 128, 129), ("f16", 9000, 40, 3000, 6000), ("bf16", 3000, 64, 0, 3000)])
def test_nan_keys_reach_every_row_that_sees_them(dt, kv, q_len, first, last):
    hkv, g, d, gs, page = 2, 4, 64, 32, 32
    q, kc, vc, table, kvs, cu = problem([kv], [q_len], hkv, g, d, gs, page, dt, 93)
    many = q_len * g > 32
    ref = attention64(q, kc, vc, table, kvs, cu, gs, d ** -0.5, 0, dt, many)
    j = torch.arange(first, last, device="cuda")
    scales = kc[1].clone()
    scales[table[0, j // page].long(), 1, j % page, 0] = float("nan")       # one group, key/value head 1
    pos = torch.arange(kv - q_len, kv, device="cuda")
    gone = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    gone[pos >= first, g:] = True
    compare(*attend(q, (kc[0], scales, kc[2]), vc, table, kvs, cu, gs, q_len), ref, gone)


@pytest.mark.parametrize("window", [2**63 - 1, 2**63 - 100, 2**62, 2**31, 2**31 - 1])
@pytest.mark.parametrize("dt,q_len", [("bf16", 3), ("f32", 150), ("f16", 150), ("bf16", 300)])
def test_windows_of_any_length(dt, q_len, window):
    """Windows beyond every position, with requests of more queries than tokens: as without one."""
    kv = [100, 260, 0, 1]
    q, kc, vc, table, kv, cu = problem(kv, [q_len] * 4, 2, 2, 64, 32, 16, dt, 99)
    out, lse = attend(q, kc, vc, table, kv, cu, 32, q_len, window=window)
    compare(out, lse, attention64(q, kc, vc, table, kv, cu, 32, 64 ** -0.5, 0, dt, q_len > 16),
            torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("M", [1, 2, 3, 8, 40])
@pytest.mark.parametrize("between", [False, True])
def test_products_with_cached_rows_right_after_an_append(M, between):
    """The cache as a weight matrix of gai4_qmv and gai4_qmm_t (which read weights before the kernels ahead of them have
    ended): codes, scales and biases of the append just before, with another call of the library between or not."""
    hkv, d, gs, page, nb = 8, 128, 64, 64, 320
    T = nb * page
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(T, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    slots = torch.randperm(T, generator=gen, device="cuda")
    kc, vc = (g4.gai4_kv_cache(nb, hkv, page, d, gs) for _ in range(2))
    x = torch.randn(M, d, generator=gen, device="cuda").bfloat16()

    def product(c):
        w = (c[0].view(-1, d // 8), c[1].view(-1, d // gs), c[2].view(-1, d // gs))
        return g4.gai4_qmv(*w, x[0], group_size=gs) if M == 1 else g4.gai4_qmm_t(*w, x, group_size=gs)

    want = []
    for i in range(2):
        g4.gai4_kv_append(rows[i], rows[1 - i], slots, kc, vc, group_size=gs)
        torch.cuda.synchronize()
        want.append((product(kc), product(vc)))
        torch.cuda.synchronize()
    for turn in range(20):
        i = turn & 1
        g4.gai4_kv_append(rows[i], rows[1 - i], slots, kc, vc, group_size=gs)
        if between:
            g4.gai4_kv_read(kc, slots[:3], group_size=gs)
        got = product(kc), product(vc)
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1]), turn


def many_rows64(q, k, v, pos, window, scale, u):
    """(out, bound) of query rows at positions pos over keys and values [kv, hkv, d] in float64, the bound as in
    kv_ref.attention64 for many rows (the score's by |k|: its keys are what the kernel multiplies)."""
    n, hq, d = q.shape
    kv, hkv = k.shape[:2]
    j = torch.arange(kv, device=q.device)
    see = j <= pos[:, None]
    if window:
        see &= j > pos[:, None] - window
    qh = q.double().unflatten(1, (hkv, hq // hkv))
    s = torch.where(see[:, None, None], scale * torch.einsum("thgd,khd->thgk", qh, k), -np.inf)
    S = abs(scale) * torch.where(see[:, None, None], torch.einsum("thgd,khd->thgk", qh.abs(), k.abs()), 0.0).amax(-1)
    p = torch.softmax(s, -1).nan_to_num(0.0)
    out, A = (torch.einsum("thgk,khd->thgd", p, x).flatten(1, 2) for x in (v, v.abs()))
    delta = (140 * 2.0**-24 + u) * S + 2.0**-21 * (1 + S)
    rel = (torch.exp(2 * delta) - 1 + 2 * u + kv * 2.0**-24).flatten(1, 2)
    return out, rel[..., None] * A + out.abs() * 2 * u + 2.0**-24


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("s,b,code", [(10000.0, 0.0, 15), (-10000.0, 30000.0, 15), (4368.0, 0.0, 15), (65504.0, 65504.0, 9),
                                      (8736.0, -65504.0, 15), (1.0, 65504.0, 15), (-65504.0, -65504.0, 12), (3000.0, 0.0, 11)])
def test_f16_groups_of_large_values(what, s, b, code):
    """Many rows: finite scales and biases whose combination is beyond binary16 (or nearly), at tokens that some rows do
    not see. These keep their result; values are computed in the others as well (keys are at most 65504)."""
    hkv, g, d, gs, page, kv, q_len, window, dt = 2, 4, 64, 32, 32, 500, 60, 200, "f16"
    q, kc, vc, table, kvs, cu = problem([kv], [q_len], hkv, g, d, gs, page, dt, 95)
    cache = [x.clone() for x in (kc if what == "k" else vc)]
    tokens = [kv - 20, kv - q_len - window + 30, kv - q_len - window]     # the last is seen by none
    for t in tokens:
        at = (int(table[0, t // page]), 1, t % page)
        cache[1][at][1], cache[2][at][1] = s, b
        cache[0][at][gs // 8] = 0x11111111 * code - (1 << 32 if code > 7 else 0)     # eight channels at `code`
    pos = torch.arange(kv - q_len, kv, device="cuda")
    hit = torch.zeros(q_len, dtype=torch.bool, device="cuda")
    for t in tokens:
        hit |= (t <= pos) & (t > pos - window)
    assert bool(hit.any()) and not bool(hit.all())
    args = (q, cache, vc) if what == "k" else (q, kc, cache)
    out, lse = attend(*args, table, kvs, cu, gs, q_len, window)
    j = torch.arange(kv, device="cuda")
    k, v = (rows64(c, table[0, j // page].long(), j % page, gs)[0] for c in args[1:])
    want, bound = many_rows64(q, k, v, pos, window, d ** -0.5, U[dt])
    check = (want.abs() + bound < 65504) & (~hit[:, None, None] if what == "k" else True)      # (outputs are binary16)
    assert bool(check[~hit].all())
    err = (out.double() - want).abs()
    assert bool((err <= bound)[check].all()), f"{int((~(err <= bound))[check].sum())} outside"


def test_f16_rows_of_the_largest_values_through_the_cache():
    """Rows that span 0 to 65504 and -65504 to 65504, appended: their groups' last code is beyond binary16."""
    hkv, d, gs, page, kv, q_len = 2, 64, 32, 32, 130, 60
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(kv, hkv, d, generator=gen, device="cuda").half() for _ in range(2))
    v[100, 1, 3], v[100, 1, 4], v[115, 1, 40], v[115, 1, 50] = 65504.0, 0.0, 65504.0, -65504.0
    v[100, 1, 5:32] = v[100, 1, 5:32].abs()
    v[100, 1, :3] = 1.0
    kc, vc = (g4.gai4_kv_cache(5, hkv, page, d, gs, torch.float16) for _ in range(2))
    g4.gai4_kv_append(k, v, torch.arange(kv, device="cuda"), kc, vc, group_size=gs)
    q = torch.randn(q_len, 8, d, generator=gen, device="cuda").half()
    out, _ = attend(q, kc, vc, i32([[0, 1, 2, 3, 4]]), [kv], [0, q_len], gs, q_len)
    j = torch.arange(kv, device="cuda")
    kk, vv = (rows64(c, j // page, j % page, gs)[0] for c in (kc, vc))
    pos = torch.arange(kv - q_len, kv, device="cuda")
    want, bound = many_rows64(q, kk, vv, pos, 0, d ** -0.5, U["f16"])
    assert float(want[pos < 100].abs().max()) < 10 and bool((want.abs() + bound < 65504).all())
    assert bool(((out.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("e", [40, 60, 100, 124])
@pytest.mark.parametrize("dt,kv,q_len,window", [("bf16", 300, 4, 0), ("f32", 300, 3, 0), ("bf16", 300, 1, 50),
                                                ("f32", 700, 4, 100), ("bf16", 5000, 4, 3000), ("f32", 400, 20, 0)])
def test_large_scales_on_tokens_that_a_row_does_not_see(dt, kv, q_len, window, e):
    """Finite value scales of 2^e, at a token that none sees and at one that only the later rows see."""
    hkv, g, d, gs, page = 2, 2, 64, 32, 32
    q, kc, vc, table, kvs, cu = problem([kv], [q_len], hkv, g, d, gs, page, dt, 97)
    scales = vc[1].clone()
    tokens = ([kv - 1] if q_len > 1 else []) + ([kv - q_len - window] if window else [])
    for t in tokens:
        scales[int(table[0, t // page]), 1, t % page, 1] = 2.0**e
    vc = (vc[0], scales, vc[2])
    out, lse = attend(q, kc, vc, table, kvs, cu, gs, q_len, window)
    want, bound, rl, lb = attention64(q, kc, vc, table, kvs, cu, gs, d ** -0.5, window, dt)
    # the row that sees such a token: eight times p s, rounded to 11 bits, where the code is 0
    if q_len > 1:
        bound[-1, g:] += 2.0 ** (e - 8)
    compare(out, lse, (want, bound, rl, lb), torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("s,b", [(2.0**126, 0.0), (2.0**125, 0.0), (2.0**127, -(2.0**127)), (2.0**124, 3.2e38), (0.5, 3.3e38)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_value_groups_at_the_end_of_the_range(dt, s, b):
    """Few rows: a group whose middle, 8 s + b, is beyond binary32 counts as infinite, and only for the rows that see
    its token; others are computed."""
    hkv, g, d, gs, page, kv, q_len, window = 2, 2, 64, 32, 32, 500, 4, 100
    q, kc, vc, table, kvs, cu = problem([kv], [q_len], hkv, g, d, gs, page, dt, 98)
    ref = attention64(q, kc, vc, table, kvs, cu, gs, d ** -0.5, window, dt)
    cache = [x.clone() for x in vc]
    tokens = [kv - 2, kv - q_len - window, kv - q_len - window + 1]
    for t in tokens:
        at = (int(table[0, t // page]), 1, t % page, 1)
        cache[1][at], cache[2][at] = s, b
    out, lse = attend(q, kc, cache, table, kvs, cu, gs, q_len, window)
    pos = torch.arange(kv - q_len, kv, device="cuda")
    hit = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    for t in tokens:
        hit[(t <= pos) & (t > pos - window), g:, gs:] = True
    assert bool(hit[2:, g:].any()) and not bool(hit[1].any())       # (the second row sees none of the three)
    want, bound, _, _ = ref
    assert bool(((out.double() - want).abs() <= bound)[~hit].all())
    if 8 * s + b > 3.4028235e38:
        assert bool(out[hit].isnan().all())
    else:
        want, bound, _, _ = attention64(q, kc, cache, table, kvs, cu, gs, d ** -0.5, window, dt)
        assert bool(((out.double() - want).abs() <= bound)[want.abs() + bound < 3.3e38].all())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,batch", [(1, 3), (40, 300)])
def test_one_key_far_above_many(dt, q_len, batch):
    """A first key that takes nearly all of the softmax and has values of zero, and thousands of others of one score,
    1.44e-7 of its probability each, whose values are one: their sum is the output. Requests share their pages, and are so
    many that most units are whole. Beside the usual bound, many rows in f16: probabilities are multiples of 2^-31 of the
    row's largest, so off by half of that for each key."""
    d, gs, page, kv = 64, 64, 64, 5033
    nb = -(-kv // page)
    q = torch.full((batch * q_len, 2, d), 1.0, dtype=DT[dt], device="cuda")
    kc, vc = (g4.gai4_kv_cache(nb, 1, page, d, gs, DT[dt]) for _ in range(2))
    kc[2][0, 0, 0] = 1.96875              # scores of 0.125 * 64 * 1.96875 = 15.75 and 0
    vc[2].fill_(1.0)
    vc[2][0, 0, 0] = 0.0
    table = torch.arange(nb, dtype=torch.int32, device="cuda").expand(batch, nb).contiguous()
    out, lse = attend(q, kc, vc, table, [kv] * batch, [q_len * i for i in range(batch + 1)], gs, q_len)
    want, bound, rl, lb = attention64(q[:q_len], kc, vc, table[:1], [kv], [0, q_len], gs, d ** -0.5, 0, dt, q_len > 16)
    if dt == "f16" and q_len > 16:
        bound = bound + kv * 2.0**-32
    assert bool(((want > 7e-4) & (want < 8e-4)).all())
    err = (out.double().view(batch, q_len, 2, d) - want).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound).max()):.3g} of the bound"
    assert bool(((lse.double().view(batch, q_len, 2) - rl).abs() <= lb).all())


@pytest.mark.parametrize("e,scale", [(100, 2.0**-103), (100, -(2.0**-104)), (90, 0.0)])
@pytest.mark.parametrize("q_len", [1, 40])
def test_extreme_queries_and_scales(q_len, e, scale):
    q, kc, vc, table, kv, cu = problem([130, 64], [q_len] * 2, 2, 4, 64, 64, 16, "bf16", 61)
    q = (q.float() * 2.0**e).bfloat16()
    out, lse = attend(q, kc, vc, table, kv, cu, 64, q_len, scale=scale)
    compare(out, lse, attention64(q, kc, vc, table, kv, cu, 64, scale, 0, "bf16", q_len > 1),
            torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda"))


def test_prompts_without_a_stated_query_length():
    """max_q_len left out: taken from the number of rows a request, so a prompt gets the kernel of many rows and single
    tokens that of few."""
    for kv, q_len, stated in (([300], [200], 200), ([300, 400], [1, 1], 1), ([90, 80], [80, 60], 70)):
        q, kc, vc, table, kv, cu = problem(kv, q_len, 2, 4, 64, 32, 32, "bf16", 103)
        a = g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=32)
        b = g4.gai4_kv_attention(q, kc, vc, table, i32(kv), i32(cu), group_size=32, max_q_len=stated)
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g,q_len,window", [(33, 9, 0), (48, 40, 100), (71, 21, 0), (300, 5, 0), (300, 1, 64), (1000, 3, 0)])
def test_many_query_heads_per_key_head(dt, g, q_len, window):
    kv = [150, 700, 3]
    q, kc, vc, table, kv, cu = problem(kv, [q_len, q_len, 1], 1, g, 64, 32, 32, dt, 101)
    out, lse = attend(q, kc, vc, table, kv, cu, 32, q_len, window)
    compare(out, lse, attention64(q, kc, vc, table, kv, cu, 32, 64 ** -0.5, window, dt, True),
            torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_a_step_of_single_tokens_and_a_prompt_as_two_calls(dt):
    """The second call has the tables and offsets of the later requests, and leaves the first one's rows alone."""
    kv, q_lens = [90, 700, 1, 400, 60], [1, 1, 1, 150, 60]
    q, kc, vc, table, kv, cu = problem(kv, q_lens, 2, 4, 64, 32, 32, dt, 105)
    q = torch.cat([q, q[:2]])          # two rows of no request
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 5.0, device="cuda")
    kvt, cut = i32(kv), i32(cu)
    g4.gai4_kv_attention(q[:3], kc, vc, table[:3], kvt[:3], cut[:4], group_size=32, max_q_len=1, out=out[:3], lse=lse[:3])
    first = out.clone(), lse.clone()
    assert bool((out[3:] == 7.0).all()) and bool((lse[3:] == 5.0).all())
    g4.gai4_kv_attention(q, kc, vc, table[3:], kvt[3:], cut[3:], group_size=32, max_q_len=150, out=out, lse=lse)
    assert torch.equal(out[:3], first[0][:3]) and torch.equal(lse[:3], first[1][:3])
    assert bool((out[-2:] == 0.0).all()) and bool((lse[-2:] == -np.inf).all())
    for many, rows in ((False, slice(0, 3)), (True, slice(3, cu[-1]))):
        want, bound, rl, lb = attention64(q[:cu[-1]], kc, vc, table, kv, cu, 32, 64 ** -0.5, 0, dt, many)
        assert bool(((out[rows].double() - want[rows]).abs() <= bound[rows]).all())
        assert bool(((lse[rows].double() - rl[rows]).abs() <= lb[rows]).all())
