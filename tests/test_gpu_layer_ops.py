"""Rotary positions, norm, e4m3 quantization and product against 64-bit references (layer_ref.py)."""
import math

import pytest
import torch

import gemm_affine_int4_gb300 as g4
from layer_ref import E4M3, TINY, U, mm64, norm64, quantize_ref, rope64, values, within

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
inf, nan = float("inf"), float("nan")


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def same(a, b):
    """Equal bit for bit, NaN for NaN."""
    a, b = a.float(), b.float()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


# ---------------------------------------------------------------- rotary positions

def positions(n, far, seed=1):
    p = torch.randint(far, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    p[:1] = 0
    p[-1:] = far - 1
    return p.cuda()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,hq,hkv,d,rot,far", [
    (1, 1, 1, 64, 64, 8), (64, 32, 8, 128, 128, 131072), (777, 7, 1, 80, 20, 4000), (5, 3, 2, 96, 24, 2 ** 31 - 1),
    (130, 16, 16, 256, 64, 10 ** 6), (33, 2, 0, 6, 2, 100), (9, 40, 8, 1024, 1024, 5000), (2000, 1, 1, 34, 34, 70000),
    (3000, 5, 2, 72, 48, 9000), (21, 4, 1, 1000, 40, 9000)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(dt, n, hq, hkv, d, rot, far, interleaved):
    qkv = rand(n, hq + 2 * hkv, d, dtype=T[dt])
    q, k, _ = qkv.split([hq, hkv, hkv], 1)
    k = k if hkv else None
    pos = positions(n, far)
    f, _ = g4.gai4_rope_inv_freq(rot)
    before = qkv.clone()
    out = g4.gai4_rope(q, k, pos, f, interleaved=interleaved, mscale=1.25)
    assert torch.equal(qkv, before)
    for x, y in zip((q, k), out):
        if x is not None:
            ref, bound = rope64(x, pos, f, 1.25, interleaved)
            within(y, ref, bound, "rope")
            assert torch.equal(y[..., rot:], x[..., rot:])
    # in place, as slices of the projection's output: the same values, and v as it was
    g4.gai4_rope(q, k, pos, f, interleaved=interleaved, mscale=1.25, q_out=q, k_out=k)
    assert torch.equal(q, out[0]) and (k is None or torch.equal(k, out[1]))
    assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])


def test_rope_odd_strides_and_offsets():
    """Rows that start on any element: every width of access."""
    n, h, d = 50, 3, 64
    pos, (f, _) = positions(n, 9000), g4.gai4_rope_inv_freq(d)
    for dt in T.values():
        for off, stride in ((0, h * d), (1, h * d + 1), (2, h * d + 2), (4, h * d + 4), (8, h * d + 8), (3, h * d + 13)):
            flat = rand(n * stride + off, dtype=dt)
            q = flat[off:].as_strided((n, h, d), (stride, d, 1), flat.storage_offset() + off)
            out = torch.empty(n * stride + off, dtype=dt, device="cuda").as_strided((n, h, d), (stride, d, 1), off)
            got, _ = g4.gai4_rope(q, None, pos, f, q_out=out)
            within(got, *rope64(q, pos, f, 1.0, False), f"offset {off}")


def test_rope_negative_positions_turn_back_and_far_ones_keep_their_angle():
    n, d = 64, 128
    f, _ = g4.gai4_rope_inv_freq(d)
    q = rand(n, 2, d)
    pos = positions(n, 2 ** 31 - 1)
    there, _ = g4.gai4_rope(q, None, pos, f)
    back, _ = g4.gai4_rope(there, None, -pos, f)
    # both turns have the same sines, off by 5 u at most, and round their products: 2 (8 u) of |a| + |b| <= 2 max
    within(back, q, 2 * 16 * 2.0 ** -24 * q.double().abs().amax(-1, keepdim=True), "there and back")
    lowest = torch.full((n,), -2 ** 31, dtype=torch.int32, device="cuda")
    within(g4.gai4_rope(q, None, lowest, f)[0], *rope64(q, lowest, f, 1.0, False), "lowest position")
    # frequencies of whole and half turns a position, above 2 pi, zero, negative, and ones that are no numbers
    fs = torch.tensor([math.pi, 2 * math.pi, 100.0, 0.0, -0.3, 1e-300, inf, nan], dtype=torch.float64, device="cuda")
    x = rand(n, 1, 16)
    pos = positions(n, 1000)
    y, _ = g4.gai4_rope(x, None, pos, fs)
    ok = [0, 1, 2, 3, 4, 5, 8, 9, 10, 11, 12, 13]
    ref, bound = rope64(x[..., ok], pos, fs[:6], 1.0, False)
    # the reference's own product position * frequency is off by half an ulp of up to 2^17
    within(y[..., ok], ref, bound + 2.0 ** -36 * x.double().abs().amax(), "odd frequencies")
    assert bool(y[..., [6, 7, 14, 15]].isnan().all())


def test_rope_keeps_infinities_and_nan_to_their_pairs():
    f, _ = g4.gai4_rope_inv_freq(16)
    x = rand(4, 1, 16)
    x[1, 0, 3], x[2, 0, 9] = nan, inf
    y, _ = g4.gai4_rope(x, None, positions(4, 50), f)
    bad = torch.zeros(4, 16, dtype=torch.bool)
    bad[1, [3, 11]] = bad[2, [1, 9]] = True
    assert torch.equal(~y[:, 0].isfinite().cpu(), bad)


# ---------------------------------------------------------------- norm

SHAPES = [(1, 1), (1, 4096), (3, 7), (64, 4096), (5, 8200), (700, 128), (701, 129), (1000, 5120), (33, 1000), (2, 32768),
          (3, 32776), (2, 100001), (400, 17), (350, 12288), (5000, 100),
          (1003, 16384), (320, 16392), (900, 511), (400, 264), (777, 1032), (1500, 5120), (3001, 520)]


def check_codes(codes, scales, y, rel, root=None):
    """e4m3 rows against y in 64 bits: the scale is off by y's own bound and two roundings, a value by half a step of
    e4m3 (2^-4 of it, 2^-10 of the scale near zero) and by y's bound. `root` [R, 1], where rows are zero: a block's
    least maximum, 2^-100, is one of y * root."""
    R, C = y.shape
    a = torch.nn.functional.pad(y.abs(), (0, -C % 128)).unflatten(1, (-1, 128)).amax(-1)
    a = torch.maximum(a, 2.0 ** -100 / root) if root is not None else a.clamp(min=2.0 ** -100)
    within(scales, a / 448, a / 448 * (rel + 3 * 2.0 ** -24), "scales")
    s = scales.double().repeat_interleave(128, 1)[:, :C]
    got = codes.double() * s
    within(got, y, torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10) + y.abs() * (rel + 4 * 2.0 ** -24), "codes")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(dt, rows, cols):
    x, r = rand(rows, cols, dtype=T[dt]), rand(rows, cols, seed=1, dtype=T[dt])
    x[:, cols // 2] *= 30
    gain = rand(cols, seed=2, dtype=T[dt])
    for residual in (None, r):
        h, y, rel = norm64(x, gain, 1e-5, residual)
        plain = g4.gai4_rms_norm(x, gain, eps=1e-5, residual=residual)
        both = g4.gai4_rms_norm(x, gain, eps=1e-5, residual=residual, fp8=True, out=torch.empty_like(x))
        only = g4.gai4_rms_norm(x, gain, eps=1e-5, residual=residual, fp8=True)
        assert plain.codes is None and only.out is None and (plain.residual is None) == (residual is None)
        within(plain.out, y, y.abs() * (rel + U[T[dt]]) + TINY[T[dt]], "norm")
        if residual is not None:
            assert torch.equal(plain.residual, (x.float() + r.float()).to(T[dt]))
            assert torch.equal(plain.residual, only.residual) and torch.equal(plain.residual, both.residual)
        check_codes(only.codes, only.scales, y, rel)
        within(both.out, y, y.abs() * (rel + U[T[dt]]) + TINY[T[dt]], "norm beside codes")
        assert torch.equal(both.scales, only.scales)
        assert torch.equal(both.codes.view(torch.uint8), only.codes.view(torch.uint8))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(9728, 520), (10001, 1024), (12345, 777), (1217, 16392), (1300, 17001)])
def test_norm_of_many_rows_into_codes(dt, rows, cols):
    """Rows enough for a warp a row: with and without residual and gain, strided, in place."""
    x, r = rand(rows, cols + 8, dtype=T[dt])[:, :cols], rand(rows, cols, seed=1, dtype=T[dt])
    x[:, cols // 2] *= 30
    x[3] = 0
    gain = rand(cols, seed=2, dtype=T[dt])
    for residual, g in ((None, gain), (r, gain), (r, None)):
        h, y, rel = norm64(x, g, 1e-5, residual, a_warp_a_row=True)
        inputs = None if residual is None else residual.clone()
        got = g4.gai4_rms_norm(x, g, eps=1e-5, residual=inputs, fp8=True, residual_out=inputs)
        check_codes(got.codes, got.scales, y, rel, root=torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5))
        if residual is not None:
            assert got.residual is inputs and torch.equal(inputs, (x.float() + r.float()).to(T[dt]))
    x[5, 7], x[6, cols - 1] = nan, inf
    got = g4.gai4_rms_norm(x, gain, eps=1e-5, fp8=True)
    v = values(got.codes[:8], got.scales[:8], 1)
    assert bool(v[5].isnan().all()) and bool(v[6, cols - 1].isnan()) and not bool(v[[0, 3, 4, 7]].isnan().any())


def test_norm_strided_rows_in_place_and_without_gain():
    for dt in T.values():
        for cols, off in ((512, 0), (512, 1), (511, 3), (40000, 8)):
            big, big2 = rand(9, 2 * cols + 16, dtype=dt), rand(9, cols + 24, seed=5, dtype=dt)
            x, r = big[:, off:off + cols], big2[:, 8:8 + cols]
            h, y, rel = norm64(x, None, 0.0, r)
            got = g4.gai4_rms_norm(x, eps=0.0, residual=r)
            within(got.out, y, y.abs() * (rel + U[dt]) + TINY[dt], f"strided {cols} {off}")
            # residual and x themselves as outputs
            a, b = x.clone(), r.clone()
            again = g4.gai4_rms_norm(a, eps=0.0, residual=b, out=a, residual_out=b)
            assert again.out is a and again.residual is b
            # (rows of another alignment may be summed in another order)
            within(a, y, y.abs() * (rel + U[dt]) + TINY[dt], f"in place {cols} {off}")
            assert torch.equal(b, got.residual)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(400, 264), (1000, 2048), (500, 16384), (700, 1001), (310, 20000)])
def test_norm_of_many_rows_in_place(dt, rows, cols):
    x, r, gain = rand(rows, cols, dtype=T[dt]), rand(rows, cols, seed=1, dtype=T[dt]), rand(cols, seed=2, dtype=T[dt])
    for residual in (None, r):
        h, y, rel = norm64(x, gain, 1e-6, residual)
        a, b = x.clone(), None if residual is None else residual.clone()
        got = g4.gai4_rms_norm(a, gain, residual=b, out=a, residual_out=b)
        assert got.out is a
        within(a, y, y.abs() * (rel + U[T[dt]]) + TINY[T[dt]], "in place")
        assert b is None or torch.equal(b, (x.float() + r.float()).to(T[dt]))


def test_norm_rows_of_zeros_and_of_no_numbers():
    x = rand(6, 300, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 5], x[3, 299], x[4] = nan, inf, 2.0 ** -126
    n = g4.gai4_rms_norm(x, eps=0.0, fp8=True, out=torch.empty_like(x))
    v = values(n.codes, n.scales, 1)
    _, y, rel = norm64(x, None, 0.0, None)
    for row in (0, 5):
        within(n.out[row], y[row], y[row].abs() * (rel + 2.0 ** -8), "rows beside")
    assert bool(n.out[2].isnan().all()) and bool(v[2].isnan().all())
    assert bool(n.out[3, 299].isnan()) and bool((n.out[3, :299] == 0).all()) and bool(v[3, 256:].isnan().all())
    z = g4.gai4_rms_norm(x[1:2], eps=1e-6, fp8=True, out=torch.empty_like(x[1:2]))
    assert bool((z.out == 0).all()) and bool((z.codes.float() == 0).all()) and bool((z.scales > 0).all())


# ---------------------------------------------------------------- e4m3 quantization

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (7, 130), (33, 14336), (129, 128), (300, 1000), (2000, 2056),
                                       (128, 8), (127, 4097), (1500, 1001), (3000, 24), (77, 300),
                                       (2500, 384), (9000, 80)])
def test_quantize(dt, rows, cols):
    x = rand(rows, cols, seed=3, dtype=T[dt]) * 2 ** torch.randint(-3, 4, (rows, 1), device="cuda").to(T[dt])
    for fn, block in ((g4.gai4_quantize_x_fp8, 1), (g4.gai4_quantize_fp8, 128)):
        codes, scales = fn(x)
        ref, ref_scales = quantize_ref(x, block)
        assert codes.dtype == E4M3 and torch.equal(scales, ref_scales)
        assert torch.equal(codes.view(torch.uint8), ref.view(torch.uint8))


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_borders(block):
    """Values midway between two codes (ties go to even), tiny and huge blocks, zeros, infinities, NaN."""
    fn = g4.gai4_quantize_x_fp8 if block == 1 else g4.gai4_quantize_fp8
    ties = torch.tensor([(m + 0.5) * 2.0 ** e / 8 for e in range(-5, 8) for m in range(8, 16)], device="cuda")
    for top in (448.0, 448.0 * 3, 448.0 * 129 / 128, 448.0 / 8192):     # scales of few bits: exact ties
        row = torch.zeros(128, device="cuda")
        row[:104] = ties * (top / 448)
        row[127] = -top
        x = row.bfloat16().float()[None]
        codes, scales = fn(x)
        ref, ref_scales = quantize_ref(x, block)
        exact = (x.double() * 448 / x.double().abs().max()).float().to(E4M3)
        assert torch.equal(codes.view(torch.uint8), ref.view(torch.uint8)) and torch.equal(scales, ref_scales)
        assert torch.equal(codes.view(torch.uint8), exact.view(torch.uint8))
    x = rand(8, 128)
    x[0], x[1], x[2], x[3] = 0, x[1] * 1e-35, x[2] * 1e37, x[3] * 2.0 ** -149
    x = x.repeat_interleave(block, 0)
    codes, scales = fn(x)
    ref, ref_scales = quantize_ref(x, block)
    assert same(codes, ref) and torch.equal(scales, ref_scales)      # (as values: the code of -0 may be that of 0)
    x = rand(6, 384).repeat_interleave(block, 0)
    x[0, 5], x[block, 200], x[2 * block, 383], x[3 * block, 0] = nan, inf, -inf, -nan
    codes, scales = fn(x)
    v = values(codes, scales, block)
    clean, clean_scales = fn(torch.where(x.isfinite(), x, 0.0))
    for r in range(6):
        for c in range(3):
            rows, cols = slice(r * block, (r + 1) * block), slice(c * 128, (c + 1) * 128)
            if (r, c) in ((0, 0), (1, 1), (2, 2), (3, 0)):
                assert bool(v[rows, cols].isnan().all())
            else:
                assert torch.equal(codes[rows, cols].view(torch.uint8), clean[rows, cols].view(torch.uint8))
                assert float(scales[r, c]) == float(clean_scales[r, c])


def test_quantize_x_strided_and_offset():
    for dt in T.values():
        big = rand(70, 1000, dtype=dt)
        for x in (big[:, 8:520], big[:, 1:900], big[::3, :640], big[5:6, 3:4]):
            codes, scales = g4.gai4_quantize_x_fp8(x)
            ref, ref_scales = quantize_ref(x, 1)
            assert torch.equal(codes.view(torch.uint8), ref.view(torch.uint8)) and torch.equal(scales, ref_scales)


# ---------------------------------------------------------------- product

def problem(M, N, K, seed=0):
    wc, ws = g4.gai4_quantize_fp8(rand(N, K, seed=seed) * (0.3 + rand(N, 1, seed=seed + 1).abs()))
    xc, xs = g4.gai4_quantize_x_fp8(rand(M, K, seed=seed + 2) * (0.3 + rand(M, 1, seed=seed + 3).abs()))
    return wc, ws, xc, xs


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 4096, 4096), (2, 129, 272), (15, 1000, 2048), (16, 128, 128), (17, 640, 1040), (32, 5120, 896),
    (33, 300, 5136), (56, 2048, 2048), (64, 512, 14336), (65, 200, 384), (100, 1111, 1616), (128, 256, 256),
    (129, 257, 144), (200, 700, 3088), (300, 1024, 2064), (513, 384, 640), (1111, 500, 1424), (2048, 1024, 512),
    (1500, 1600, 512), (1500, 1601, 528), (1537, 1540, 144), (2304, 2048, 384), (2300, 2041, 272), (700, 5000, 2064)])
def test_mm(dt, M, N, K):
    p = problem(M, N, K)
    out = g4.gai4_fp8_mm_t(*p, dtype=T[dt])
    assert g4.gai4_last_device_status() == 0
    ref, bound = mm64(*p, T[dt])
    within(out, ref, bound, f"mm {M} {N} {K}")
    assert torch.equal(out, g4.gai4_fp8_mm_t(*p, dtype=T[dt]))       # bit for bit


@pytest.mark.parametrize("M,N", [(1, 400), (40, 400), (128, 400), (400, 400), (1500, 1700), (2304, 2048)])
def test_mm_every_block_has_its_scales(M, N):
    """Scales that differ by powers of two from block to block, of rows and of columns: a wrong one is out by half."""
    K = 1200
    g = torch.Generator(device="cuda").manual_seed(9)
    wc, _, xc, _ = problem(M, N, K)
    ws = 2.0 ** torch.randint(-6, 7, (-(-N // 128), 10), generator=g, device="cuda")
    xs = 2.0 ** torch.randint(-6, 7, (M, 10), generator=g, device="cuda")
    out = g4.gai4_fp8_mm_t(wc, ws, xc, xs, dtype=torch.float32)
    within(out, *mm64(wc, ws, xc, xs, torch.float32), "scales")


@pytest.mark.parametrize("M,N", [(3, 300), (50, 300), (120, 300), (700, 300), (1500, 1700), (2304, 2048)])
def test_mm_exact_small_integers(M, N):
    """Codes of small integers and scales of one: every sum is a whole number, exactly."""
    K = 1136
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float()
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float()
    ones = lambda r: torch.ones(r, 9, device="cuda")  # noqa: E731
    out = g4.gai4_fp8_mm_t(w.to(E4M3), ones(-(-N // 128)), x.to(E4M3), ones(M), dtype=torch.float32)
    assert torch.equal(out.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M,N", [(5, 200), (300, 200), (1500, 1700), (2304, 2048)])
def test_mm_not_a_number_stays_in_its_row_and_column(M, N):
    K = 512
    wc, ws, xc, xs = problem(M, N, K)
    clean = g4.gai4_fp8_mm_t(wc, ws, xc, xs)
    wc.view(torch.uint8)[7, 300] = 0x7F
    xc.view(torch.uint8)[2, 5] = 0xFF
    out = g4.gai4_fp8_mm_t(wc, ws, xc, xs)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 7] = True, True
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("M,N", [(1, 333), (60, 333), (128, 336), (333, 333), (1500, 1701), (1500, 1704), (2300, 2048)])
def test_mm_writes_its_rows_only(M, N):
    K = 256
    p = problem(M, N, K)
    room = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    g4.gai4_fp8_mm_t(*p, out=room[1:M + 1])
    assert bool((room[0] == 7).all()) and bool((room[M + 1] == 7).all())
    assert torch.equal(room[1:M + 1], g4.gai4_fp8_mm_t(*p))


# ---------------------------------------------------------------- empty calls, streams, graphs, a run of them

def test_no_rows():
    f, _ = g4.gai4_rope_inv_freq(64)
    none = torch.empty(0, 2, 64, device="cuda")
    q, k = g4.gai4_rope(none, none, torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert q.shape == k.shape == (0, 2, 64)
    x = torch.empty(0, 256, device="cuda")
    n = g4.gai4_rms_norm(x, fp8=True)
    assert n.codes.shape == (0, 256) and n.scales.shape == (0, 2)
    c, s = g4.gai4_quantize_x_fp8(x)
    wc, ws = g4.gai4_quantize_fp8(rand(64, 256))
    assert g4.gai4_fp8_mm_t(wc, ws, c, s).shape == (0, 64)


class Step:
    """norm -> product -> rotary positions -> append, attention -> quantization -> product."""
    H, HQ, HKV, D, PAGE = 512, 8, 2, 64, 16

    def __init__(self, tokens, seed=0):
        o = self.HQ * self.D
        self.w_qkv = g4.gai4_quantize_fp8(rand((self.HQ + 2 * self.HKV) * self.D, self.H, seed=seed) * self.H ** -0.5)
        self.w_out = g4.gai4_quantize_fp8(rand(self.H, o, seed=seed + 1) * o ** -0.5)
        self.gain = (1 + 0.1 * rand(self.H, seed=seed + 2)).bfloat16()
        self.x, self.r = rand(tokens, self.H, seed=seed + 3, dtype=torch.bfloat16), rand(tokens, self.H, seed=seed + 4).bfloat16()
        self.f, self.mscale = g4.gai4_rope_inv_freq(self.D, scaling="yarn", factor=4.0, original_len=64)
        blocks = -(-tokens // self.PAGE)
        self.kc, self.vc = (g4.gai4_kv_cache(blocks, self.HKV, self.PAGE, self.D, 32) for _ in range(2))
        ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.free = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda"), ints(*range(blocks))
        self.plan = g4.gai4_kv_plan(ints(0), ints(tokens), self.table, self.free, ints(blocks), self.PAGE, tokens)

    def run(self):
        n = g4.gai4_rms_norm(self.x, self.gain, residual=self.r, fp8=True)
        qkv = g4.gai4_fp8_mm_t(*self.w_qkv, n.codes, n.scales).unflatten(1, (-1, self.D))
        q, k, v = qkv.split([self.HQ, self.HKV, self.HKV], 1)
        g4.gai4_rope(q, k, self.plan.positions, self.f, mscale=self.mscale, q_out=q, k_out=k)
        g4.gai4_kv_append(k, v, self.plan.slots, self.kc, self.vc, group_size=32)
        o = g4.gai4_kv_attention(q, self.kc, self.vc, self.table, self.plan.kv_lens, self.plan.cu_q, group_size=32,
                                 max_q_len=self.x.shape[0])
        c, s = g4.gai4_quantize_x_fp8(o.flatten(1))
        return n.residual, q, k, o, g4.gai4_fp8_mm_t(*self.w_out, c, s)


@pytest.mark.parametrize("tokens", [3, 70, 200])
def test_a_layer(tokens):
    """Each operator of the run against its reference, on what the one before it gave."""
    st = Step(tokens)
    residual, q, k, o, out = st.run()
    h, y, rel = norm64(st.x, st.gain, 1e-6, st.r)
    n = g4.gai4_rms_norm(st.x, st.gain, residual=st.r, fp8=True)
    check_codes(n.codes, n.scales, y, rel)
    assert torch.equal(residual, n.residual)
    qkv = g4.gai4_fp8_mm_t(*st.w_qkv, n.codes, n.scales)
    within(qkv, *mm64(*st.w_qkv, n.codes, n.scales, torch.bfloat16), "qkv")
    rows = qkv.unflatten(1, (-1, st.D))
    assert torch.equal(st.plan.positions, torch.arange(tokens, dtype=torch.int32, device="cuda"))
    within(q, *rope64(rows[:, :st.HQ], st.plan.positions, st.f, st.mscale, False), "q")
    within(k, *rope64(rows[:, st.HQ:st.HQ + st.HKV], st.plan.positions, st.f, st.mscale, False), "k")
    c, s = quantize_ref(o.flatten(1), 1)
    within(out, *mm64(*st.w_out, c, s, torch.bfloat16), "out")
    assert g4.gai4_last_device_status() == 0


def test_a_layer_on_a_stream_and_in_a_graph():
    st = Step(70)
    want = st.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = st.run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = st.run()
    other = rand(70, st.H, seed=40, dtype=torch.bfloat16)
    x = st.x.clone()
    for value, expect in ((other, None), (x, want)):
        st.x.copy_(value)
        graph.replay()
        torch.cuda.synchronize()
        if expect is not None:
            assert all(torch.equal(a, b) for a, b in zip(expect, got))
        else:
            assert not torch.equal(got[-1], want[-1])


def test_two_streams_at_once():
    """Products of both kernels side by side: neither waits for the other's tensor memory for good."""
    small, large = problem(9, 2000, 4096), problem(1500, 1700, 2048, seed=7)
    want = [g4.gai4_fp8_mm_t(*p) for p in (small, large)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, p in enumerate((small, large)):
            got[i].append(g4.gai4_fp8_mm_t(*p, stream=streams[i]))
    torch.cuda.synchronize()
    assert g4.gai4_last_device_status() == 0
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def test_stream_argument():
    st = torch.cuda.Stream()
    x = rand(40, 1024, dtype=torch.float16)
    f, _ = g4.gai4_rope_inv_freq(64)
    torch.cuda.synchronize()
    n = g4.gai4_rms_norm(x, fp8=True, stream=st)
    c, s = g4.gai4_quantize_x_fp8(x, stream=st)
    wc, ws = g4.gai4_quantize_fp8(x, stream=st)
    y = g4.gai4_fp8_mm_t(wc, ws, c, s, stream=st)
    q, _ = g4.gai4_rope(x.view(40, 16, 64), None, torch.arange(40, dtype=torch.int32, device="cuda"), f, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y, g4.gai4_fp8_mm_t(wc, ws, c, s)) and torch.equal(c.view(torch.uint8), g4.gai4_quantize_x_fp8(x)[0].view(torch.uint8))
    assert torch.equal(n.scales, g4.gai4_rms_norm(x, fp8=True).scales)
    assert torch.equal(q, g4.gai4_rope(x.view(40, 16, 64), None, torch.arange(40, dtype=torch.int32, device="cuda"), f)[0])


def test_beside_products_of_4_bit_weights():
    """On two streams, in turn with kernels that take tensor memory too (4-bit weights, 16 and 300 rows)."""
    products = [problem(M, 1024, 2048, seed=M) for M in (1, 20, 50, 120, 1500)]
    w4 = g4.gai4_quantize(rand(4096, 2048) * 0.02, 4, 64, torch.bfloat16)
    rows = [rand(M, 2048, seed=M, dtype=torch.bfloat16) for M in (16, 300)]

    def step(i, stream=None):
        p, x = products[i % len(products)], rows[i % 2]
        return g4.gai4_fp8_mm_t(*p, stream=stream), g4.gai4_qmm_t(*w4, x, stream=stream)

    want = [step(i) for i in range(10)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [(i % 10, step(i % 10, streams[(i // 3) % 2])) for i in range(120)]
    torch.cuda.synchronize()
    assert g4.gai4_last_device_status() == 0
    assert all(torch.equal(a, b) for i, y in got for a, b in zip(want[i], y))


def inside(shape, dtype, before):
    """A contiguous tensor within a buffer of bytes 0x5a, and a check of what lies around it."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = math.prod(shape) * size
    room = torch.full((before + n + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    t = room[before:before + n].view(dtype).view(shape)
    return t, lambda: bool((room[:before] == 0x5a).all()) and bool((room[before + n:] == 0x5a).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("before", [64, 12])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 129), (5, 1000), (700, 1000), (700, 777), (2, 17001), (300, 64)])
def test_nothing_is_written_around_the_outputs(dt, before, rows, cols):
    x, r = rand(rows, cols, seed=1, dtype=T[dt]), rand(rows, cols, seed=2, dtype=T[dt])
    blocks = (cols + 127) // 128
    made = [inside((rows, cols), T[dt], before), inside((rows, cols), T[dt], before), inside((rows, cols), E4M3, before),
            inside((rows, blocks), torch.float32, before)]
    out, h, codes, scales = (t for t, _ in made)
    want = g4.gai4_rms_norm(x, residual=r, fp8=True, out=torch.empty_like(x))
    g4.gai4_rms_norm(x, residual=r, fp8=True, out=out, residual_out=h, codes=codes, scales=scales)
    assert all(check() for _, check in made)
    assert same(h, want.residual)
    g4.gai4_quantize_x_fp8(x, codes=codes, scales=scales)
    assert all(check() for _, check in made)
    c, s = g4.gai4_quantize_x_fp8(x)
    assert same(codes, c) and same(scales, s)
    ws, wcheck = inside(((rows + 127) // 128, blocks), torch.float32, before)
    g4.gai4_quantize_fp8(x, codes=codes, scales=ws)
    assert wcheck() and all(check() for _, check in made)
    c, s = g4.gai4_quantize_fp8(x)
    assert same(codes, c) and same(ws, s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("before", [64, 12])
@pytest.mark.parametrize("n,hq,hkv,d,rot", [(1, 1, 1, 2, 2), (3, 3, 1, 33, 32), (1000, 5, 2, 80, 40), (9, 2, 1, 1024, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_writes_its_rows_only(dt, before, n, hq, hkv, d, rot, interleaved):
    q, k = rand(n, hq, d, seed=3, dtype=T[dt]), rand(n, hkv, d, seed=4, dtype=T[dt])
    f, _ = g4.gai4_rope_inv_freq(rot)
    p = positions(n, 1000)
    (qo, qcheck), (ko, kcheck) = inside((n, hq, d), T[dt], before), inside((n, hkv, d), T[dt], before)
    g4.gai4_rope(q, k, p, f, interleaved=interleaved, q_out=qo, k_out=ko)
    assert qcheck() and kcheck()
    want = g4.gai4_rope(q, k, p, f, interleaved=interleaved)
    assert same(qo, want[0]) and same(ko, want[1])


def test_offsets_beyond_32_bits():
    """Tensors of 2254 million elements: the last rows are those of a call on them alone."""
    rows, cols, tail = 550400, 4096, 12800
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-tail:] = rand(tail, cols, dtype=torch.bfloat16)
    last = x[-tail:].clone()
    for kw in (dict(fp8=True), dict(fp8=False), dict(fp8=True, out=True)):
        big, small = (g4.gai4_rms_norm(t, residual=t, fp8=kw["fp8"], out=torch.empty_like(t) if kw.get("out") else None)
                      for t in (x, last))
        for a, b in zip(big, small):
            assert (a is None) == (b is None)
            assert a is None or same(a[-tail:], b)
        del big, small, a, b
    p = torch.arange(rows, dtype=torch.int32, device="cuda")
    f, _ = g4.gai4_rope_inv_freq(128)
    q, k = x.view(rows, 32, 128).split([28, 4], 1)
    qo, ko = g4.gai4_rope(q, k, p, f)
    want = g4.gai4_rope(*last.view(tail, 32, 128).split([28, 4], 1), p[-tail:].clone(), f)
    assert same(qo[-tail:], want[0]) and same(ko[-tail:], want[1])
    del qo, ko, want
    wc, ws = g4.gai4_quantize_fp8(x)
    c, s = g4.gai4_quantize_fp8(last)
    assert same(wc[-tail:], c) and same(ws[-tail // 128:], s)
    del wc
    xc, xs = g4.gai4_quantize_x_fp8(x)
    c, s = g4.gai4_quantize_x_fp8(last)
    assert same(xc[-tail:], c) and same(xs[-tail:], s)
    del x
    for n in (4096, 4097):   # (rows of outputs on 16-byte boundaries, and not)
        w = g4.gai4_quantize_fp8(rand(n, cols, seed=n) * 0.02)
        y = g4.gai4_fp8_mm_t(*w, xc, xs)
        assert same(y[-tail:], g4.gai4_fp8_mm_t(*w, c, s))
        del y


@pytest.mark.parametrize("M", [1, 100, 300])
def test_weights_beyond_32_bits(M):
    """Small integers, so that every order of additions gives the same."""
    N, K, tail = 550400, 4096, 1280

    def ints(n, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randint(-2, 3, (n, K), generator=g, device="cuda").to(E4M3)

    w = torch.zeros(N, K, dtype=E4M3, device="cuda")
    w[-tail:] = ints(tail, 1)
    ws = torch.ones(N // 128, K // 128, device="cuda")
    x, xs = ints(M, 2), torch.ones(M, K // 128, device="cuda")
    y = g4.gai4_fp8_mm_t(w, ws, x, xs, dtype=torch.float32)
    assert torch.equal(y[:, -tail:], x.float() @ w[-tail:].float().t()) and not bool(y[:, :-tail].any())


def test_refused_on_the_gpu():
    """What only the library's entry refuses, its types, and outputs that do not fit; the next call works."""
    x = rand(6, 256, dtype=torch.bfloat16)
    c, s = g4.gai4_quantize_x_fp8(x)
    w = g4.gai4_quantize_fp8(rand(128, 256))
    f, _ = g4.gai4_rope_inv_freq(64)
    p = torch.arange(6, dtype=torch.int32, device="cuda")
    q = x.view(6, 4, 64)
    with pytest.raises(g4.Gai4Error, match="gai4_rms_norm"):
        g4.gai4_rms_norm(x, eps=-1.0)
    with pytest.raises(g4.Gai4Error, match="gai4_rope"):
        g4.gai4_rope(q, q[:, :2], p, f, q_out=q, k_out=q[:, 2:])     # k's rows where q's are written
    with pytest.raises(g4.Gai4Error, match="gai4_fp8_mm_t"):
        narrow = g4.gai4_quantize_fp8(rand(128, 200)), g4.gai4_quantize_x_fp8(x[:, :200])
        g4.gai4_fp8_mm_t(*narrow[0], *narrow[1])                      # K a multiple of 16
    for bad in (lambda: g4.gai4_rms_norm(x.double()), lambda: g4.gai4_quantize_x_fp8(x.int()),
                lambda: g4.gai4_fp8_mm_t(*w, c, s, dtype=torch.float64),
                lambda: g4.gai4_fp8_mm_t(*w, c, s, out=torch.empty(6, 127, device="cuda")),
                lambda: g4.gai4_fp8_mm_t(*w, c, s.cpu()), lambda: g4.gai4_rope(q, None, p.cpu(), f),
                lambda: g4.gai4_rms_norm(x, out=torch.empty(6, 512, device="cuda", dtype=x.dtype)[:, ::2]),
                lambda: g4.gai4_rms_norm(x, fp8=True, codes=torch.empty(6, 256, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        g4.gai4_rms_norm(x, eps="small")
    assert same(g4.gai4_quantize_x_fp8(x.clone().requires_grad_())[0], c)
    assert same(g4.gai4_fp8_mm_t(w[0].view(torch.uint8), w[1], c.view(torch.uint8), s), g4.gai4_fp8_mm_t(*w, c, s))


def test_calls_from_several_threads():
    import threading
    x = rand(48, 4096, dtype=torch.bfloat16)
    w = g4.gai4_quantize_fp8(rand(512, 4096) * 0.02)
    want = g4.gai4_fp8_mm_t(*w, *g4.gai4_quantize_x_fp8(x))
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in range(4)]

    def work(stream):
        with torch.cuda.stream(stream):
            for _ in range(200):
                y = g4.gai4_fp8_mm_t(*w, *g4.gai4_quantize_x_fp8(x))
            stream.synchronize()
            got.append(y)

    threads = [threading.Thread(target=work, args=(s,)) for s in streams]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4 and all(torch.equal(y, want) for y in got)
