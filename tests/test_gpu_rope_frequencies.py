"""Rotary positions at any frequency and any position: angles from whole numbers, whose turns are taken off exactly."""
import math

import pytest
import torch

import gemm_affine_int4_gb300 as g4
from layer_ref import TINY, U, u, within

pytestmark = pytest.mark.gpu
BITS = 400   # of 1 / (2 pi): 2^53 times 2^31 has 84 before the point


def _inverse_turn():
    def arctan(n):   # of 1 / n
        total, term, k = 0, (1 << BITS) // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return (1 << (2 * BITS)) // (8 * (4 * arctan(5) - arctan(239)))


INVERSE_TURN = _inverse_turn()


def angle(position, frequency):
    """position * frequency modulo a turn, -pi to pi, good to 2^-50."""
    n, d = frequency.as_integer_ratio()
    turns = (position * n * INVERSE_TURN << 64) // d & (1 << (BITS + 64)) - 1
    return math.ldexp((turns >> (BITS - 53 + 64)) - (1 << 53 if turns >> (BITS + 63) else 0), -53) * 2 * math.pi


FREQUENCIES = [1.0, 1.9999, 2.0, 3.7, math.pi, 100.0, 12345.678, -1e5, 1e6 / 3, 2.0 ** 30 + 0.5, 1e12 / 7, -2.0 ** 51 / 3,
               2.0 ** 52 - 1, 2.0 ** 52 + 1, 2.0 ** 53 - 1, 5e-324, 1e-310, -1e-9, 0.7]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_any_frequency(dt, interleaved):
    half = len(FREQUENCIES)
    p = [0, 1, 2, 3, 1000, 65537, 999999937, 2 ** 31 - 1, 2 ** 31 - 2, -1, -12345, -2 ** 31, 1 << 30, 2000000011]
    p += torch.randint(-2 ** 31, 2 ** 31, (50,), generator=torch.Generator().manual_seed(2)).tolist()
    x = torch.randn(len(p), 2, 2 * half, generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    f = torch.tensor(FREQUENCIES, dtype=torch.float64, device="cuda")
    got, _ = g4.gai4_rope(x, None, torch.tensor(p, dtype=torch.int32, device="cuda"), f, interleaved=interleaved)
    t = torch.tensor([[angle(i, v) for v in FREQUENCIES] for i in p], dtype=torch.float64, device="cuda")
    c, s = t.cos()[:, None], t.sin()[:, None]
    r = x.double()
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y = (a * c - b * s, b * c + a * s)
    # as in layer_ref.rope64: sine and cosine, the magnitude, two products and their sum, and a fraction of a turn
    m = 8 * u * (a.abs() + b.abs())
    y, m = (torch.stack(v, -1).flatten(-2) if interleaved else torch.cat(v, -1) for v in (y, (m, m)))
    within(got, y, m * (1 + U[dt]) + U[dt] * y.abs() + TINY[dt], "any frequency")


def test_what_does_not_tell_an_angle():
    f = torch.tensor([2.0 ** 53, -2.0 ** 53, 1e17, 1.7e308, math.inf, -math.inf, math.nan, 0.5], dtype=torch.float64, device="cuda")
    x = torch.ones(3, 1, 16, device="cuda")
    y, _ = g4.gai4_rope(x, None, torch.tensor([0, 1, -7], dtype=torch.int32, device="cuda"), f)
    assert bool(y[..., :7].isnan().all()) and bool(y[..., 8:15].isnan().all()) and bool(y[..., [7, 15]].isfinite().all())
