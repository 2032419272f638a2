"""The operators around the attention without a GPU: frequencies, refusals before anything is launched."""
import ctypes
import math

import pytest
import torch

import gemm_affine_int4_gb300 as g4

P = ctypes.c_void_p
A, B, C, D = (P(0x100000000 * i) for i in (1, 2, 3, 4))


# ---------------------------------------------------------------- frequencies

def freqs(*a, **k):
    f, m = g4.gai4_rope_inv_freq(*a, device="cpu", **k)
    return f.tolist(), m


def test_plain_frequencies():
    f, m = freqs(128)
    assert m == 1.0 and f[0] == 1.0
    for i, x in enumerate(f):
        assert math.isclose(x, 10000.0 ** (-2 * i / 128), rel_tol=1e-14)


def test_scaled_frequencies():
    plain, _ = freqs(64, base=5e5)
    f, m = freqs(64, base=5e5, scaling="linear", factor=4.0)
    assert m == 1.0 and all(math.isclose(4 * x, y, rel_tol=1e-14) for x, y in zip(f, plain))
    # the base raised: the fastest pair stays, the slowest is divided by the factor
    f, m = freqs(64, base=5e5, scaling="ntk", factor=4.0)
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 4, rel_tol=1e-12)
    # turns over the original length: more than `high` kept, fewer than `low` divided
    f, m = freqs(64, base=5e5, scaling="smooth", factor=8.0, original_len=8192, low=1.0, high=4.0)
    assert m == 1.0
    for x, y in zip(f, plain):
        turns = 8192 * y / (2 * math.pi)
        want = y if turns >= 4 else y / 8 if turns <= 1 else y * (turns - 1) / 3 + y / 8 * (4 - turns) / 3
        assert math.isclose(x, want, rel_tol=1e-12)
    f, m = freqs(64, base=5e5, scaling="yarn", factor=8.0, original_len=8192)
    assert math.isclose(m, 0.1 * math.log(8.0) + 1, rel_tol=1e-7)
    for i, (x, y) in enumerate(zip(f, plain)):
        turns = 8192 * y / (2 * math.pi)
        assert y / 8 * (1 - 1e-12) <= x <= y
        if turns > 32:
            assert math.isclose(x, y, rel_tol=1e-12)
        if i > 0:
            assert x <= f[i - 1]
    assert math.isclose(f[-1], plain[-1] / 8, rel_tol=1e-12)
    # a factor of one changes nothing
    for s in ("linear", "ntk", "yarn", "smooth"):
        f, m = freqs(64, base=5e5, scaling=s, factor=1.0, original_len=100)
        assert m == 1.0 and all(math.isclose(x, y, rel_tol=1e-14) for x, y in zip(f, plain))
    assert freqs(2, scaling="ntk", factor=4.0) == ([1.0], 1.0)


@pytest.mark.parametrize("rot,base,factor,length,low,high", [
    (64, 5e5, 8.0, 8192, 1.0, 32.0), (128, 1e4, 4.0, 4096, 1.0, 32.0), (32, 1e4, 40.0, 4096, 2.0, 17.5), (128, 1e6, 2.0, 32768, 0.5, 64.0),
    (20, 150.0, 16.0, 300, 1.0, 8.0), (64, 1e4, 8.0, 20, 1.0, 32.0), (64, 100.0, 8.0, 1e6, 1.0, 32.0)])
def test_yarn_between_the_ends_of_its_ramp(rot, base, factor, length, low, high):
    """The ramp is linear in the pair's number, from the last pair of at least `high` turns (the first at least) to the
    first of at most `low` (or rot - 1), as if there were that many pairs."""
    f, _ = freqs(rot, base=base, scaling="yarn", factor=factor, original_len=length, low=low, high=high)
    turns = [length * base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot)]
    first = max([i for i in range(rot) if turns[i] >= high], default=0)
    last = min([i for i in range(rot) if turns[i] <= low], default=rot - 1)
    inside = 0
    for i, x in enumerate(f):
        divided = min(max((i - first) / (last - first), 0.0), 1.0) if last > first else float(i > first)
        inside += 0 < divided < 1
        plain = base ** (-2 * i / rot)
        assert math.isclose(x, plain / factor * divided + plain * (1 - divided), rel_tol=1e-12), i
    assert inside > 0 or length == 1e6


@pytest.mark.parametrize("change,status", [
    (dict(f=None), 1), (dict(m=None), 1), (dict(rot=0), 1), (dict(rot=63), 1), (dict(base=1.0), 1),
    (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(how=5), 2), (dict(how=-1), 2),
    (dict(how=1, factor=0.5), 1), (dict(how=1, factor=float("inf")), 1), (dict(how=3, length=0.0), 1),
    (dict(how=4, length=float("nan")), 1), (dict(how=3, low=0.0), 1), (dict(how=3, low=8.0, high=8.0), 1),
    (dict(how=0, factor=0.0), 0)])
def test_frequency_refusals(change, status):
    buf, m = (ctypes.c_double * 64)(), ctypes.c_float()
    a = dict(f=ctypes.addressof(buf), m=ctypes.addressof(m), rot=64, base=10000.0, how=0, factor=2.0, length=100.0,
             low=1.0, high=32.0)
    a.update(change)
    assert g4.lib().gai4_rope_inv_freq(*a.values()) == status


# ---------------------------------------------------------------- refusals

def rope(**c):
    a = dict(q=A, qs=1024, qo=B, qos=1024, k=C, ks=256, ko=D, kos=256, pos=A, f=A, m=1.0, dt=2, n=4, hq=8, hkv=2, d=128,
             rot=128, il=0)
    a.update(c)
    return g4.lib().gai4_rope(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(f=None), 1),
    (dict(qs=1023), 1), (dict(qos=0), 1), (dict(ks=255), 1), (dict(kos=-1), 1), (dict(qs=1 << 59), 1), (dict(n=(1 << 31) - 1, qs=1 << 40), 1), (dict(n=-1), 1),
    (dict(n=1 << 31), 1), (dict(hq=0, hkv=0), 1), (dict(hq=-1), 1), (dict(hkv=1 << 20), 1), (dict(rot=0), 1),
    (dict(rot=63), 1), (dict(rot=130), 1), (dict(d=0), 1), (dict(d=2048, qs=1 << 20, qos=1 << 20), 2), (dict(dt=3), 2),
    (dict(q=P(0x100000001)), 3), (dict(dt=0, ko=P(0x400000002)), 3), (dict(pos=P(0x10002)), 3), (dict(f=P(0x10004)), 3),
    # rows written over other rows
    (dict(qo=P(0x100000010)), 1), (dict(qo=A, qos=2048), 1), (dict(ko=A), 1), (dict(qo=C), 1), (dict(ko=B), 1),
    (dict(qs=1536, qos=1536, qo=A, k=P(0x100000000 + 1024), ks=1536, ko=D), 1),
    (dict(n=0), 0), (dict(n=0, q=None, qo=None, k=None, ko=None, pos=None, f=None), 0)])
def test_rope_refusals(change, status):
    assert rope(**change) == status


def norm(**c):
    a = dict(x=A, xs=512, r=B, rs=512, g=C, out=D, ro=P(0x500000000), codes=P(0x600000000), scales=P(0x700000000), dt=2,
             rows=4, cols=512, eps=1e-6)
    a.update(c)
    return g4.lib().gai4_rms_norm(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(out=None, ro=None, codes=None, scales=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(xs=511), 1), (dict(rs=1), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(cols=0), 1),
    (dict(cols=1 << 31), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(dt=9), 2), (dict(x=P(0x100000001)), 3), (dict(dt=0, g=P(0x300000002)), 3), (dict(scales=P(0x700000002)), 3),
    (dict(rows=1 << 30, xs=1 << 31), 1), (dict(out=D, ro=D), 1), (dict(out=P(0x100000000 + 64)), 1), (dict(ro=B, rs=600), 1), (dict(rows=0), 0),
    (dict(rows=0, x=None), 0)])
def test_norm_refusals(change, status):
    assert norm(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(xs=255), 1), (dict(xs=1 << 60), 1), (dict(M=-1), 1), (dict(K=0), 1),
    (dict(dt=-1), 2), (dict(x=P(0x100000001)), 3), (dict(s=P(0x10001)), 3), (dict(M=0), 0)])
def test_quantize_x_refusals(change, status):
    a = dict(x=A, xs=256, c=B, s=C, dt=1, M=3, K=256)
    a.update(change)
    assert g4.lib().gai4_quantize_x_fp8(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(w=None), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(N=0), 1), (dict(N=65535 * 128 + 1), 1), (dict(K=0), 1),
    (dict(dt=4), 2), (dict(w=P(0x100000002)), 3)])
def test_quantize_refusals(change, status):
    a = dict(w=A, c=B, s=C, dt=0, N=3, K=256)
    a.update(change)
    assert g4.lib().gai4_quantize_fp8(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(w=None), 1), (dict(ws=None), 1), (dict(x=None), 1), (dict(xs=None), 1), (dict(out=None), 1), (dict(M=-1), 1),
    (dict(N=0), 1), (dict(K=0), 1), (dict(K=24), 2), (dict(dt=3), 2), (dict(w=P(0x10008)), 3), (dict(x=P(0x10001)), 3),
    (dict(out=P(0x10001)), 3), (dict(dt=0, out=P(0x10002)), 3), (dict(xs=P(0x10002)), 3), (dict(N=1 << 31), 1),
    (dict(M=0), 0), (dict(M=0, x=None, out=None), 0)])
def test_mm_refusals(change, status):
    a = dict(w=A, ws=A, x=A, xs=A, out=A, dt=2, M=3, N=64, K=256)
    a.update(change)
    assert g4.lib().gai4_fp8_mm_t(*a.values(), None) == status


def test_binding_refuses_wrong_shapes():
    x, f = torch.zeros(3, 2, 64), torch.zeros(32, dtype=torch.float64)
    pos = torch.zeros(3, dtype=torch.int32)
    bad = [
        lambda: g4.gai4_rope(x, x, pos, f),                                        # not on a GPU
        lambda: g4.gai4_rope(x, x, pos.long(), f), lambda: g4.gai4_rope(x, x, pos[:2], f),
        lambda: g4.gai4_rope(x, x[:2], pos, f), lambda: g4.gai4_rope(x, x, pos, f.float()),
        lambda: g4.gai4_rope(x, x.half(), pos, f), lambda: g4.gai4_rope(x.transpose(0, 1), None, pos[:2], f),
        lambda: g4.gai4_rope_inv_freq(64, scaling="other", device="cpu"),
        lambda: g4.gai4_rms_norm(x[0]), lambda: g4.gai4_rms_norm(x[0], x[0, 0, :3]),
        lambda: g4.gai4_rms_norm(x[0], residual=x[1, :1]), lambda: g4.gai4_rms_norm(x[0], out=x[1].half()),
        lambda: g4.gai4_rms_norm(x[0].t()), lambda: g4.gai4_rms_norm(x[0], codes=x[0]),
        lambda: g4.gai4_quantize_x_fp8(x[0]), lambda: g4.gai4_quantize_fp8(x[0]),
        lambda: g4.gai4_quantize_x_fp8(x[0], scales=torch.zeros(2, 2)),
    ]
    c, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(4, 2)
    bad += [lambda: g4.gai4_fp8_mm_t(c, s, c, s), lambda: g4.gai4_fp8_mm_t(c, s[:1], c, s[:3]),
            lambda: g4.gai4_fp8_mm_t(c, s[:1], c[:, :128], s), lambda: g4.gai4_fp8_mm_t(c.float(), s[:1], c, s),
            lambda: g4.gai4_fp8_mm_t(c, s[:1].half(), c, s)]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_a_refused_call_raises_the_librarys_error():
    with pytest.raises(g4.Gai4Error):
        g4.gai4_rope_inv_freq(64, base=0.5, device="cpu")


def test_binding_names_what_it_was_given():
    with pytest.raises(TypeError):
        g4.gai4_quantize_x_fp8(None)
    with pytest.raises(TypeError):
        g4.gai4_fp8_mm_t(3, 4, 5, 6)
    with pytest.raises(ValueError, match="one CUDA device"):
        g4.gai4_rms_norm(torch.zeros(2, 3))
    with pytest.raises(ValueError, match="columns contiguous"):
        g4.gai4_rms_norm(torch.zeros(2, 3, 4))


@pytest.mark.parametrize("change,status", [
    (dict(status=None), 1), (dict(withheld=-1), 1), (dict(withheld=16), 1), (dict(blocks=-1), 1), (dict(limit=0), 1),
    (dict(limit=4000000001), 1), (dict(status=P(0x10002)), 3), (dict(w=None), 1), (dict(K=24), 2), (dict(M=0), 0)])
def test_withheld_loads_refusals(change, status):
    a = dict(w=A, ws=A, x=A, xs=A, out=A, dt=2, M=3, N=64, K=256, withheld=1, blocks=0, limit=1000, status=A)
    a.update(change)
    assert g4.lib().gai4_check_fp8_mm_wait(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [(dict(M=0), 1), (dict(N=0), 1), (dict(K=24), 2), (dict(dt=3), 2), (dict(a=None), 1),
                                           (dict(b=None), 1), (dict(c=None), 1), (dict(M=1 << 31), 1)])
def test_product_plan_refusals(change, status):
    i, j, k = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    a = dict(M=3, N=64, K=256, dt=2, a=ctypes.byref(i), b=ctypes.byref(j), c=ctypes.byref(k))
    a.update(change)
    assert g4.lib().gai4_fp8_mm_t_plan(*a.values()) == status
