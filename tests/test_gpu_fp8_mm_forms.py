"""The e4m3 product in each of its forms (tokens at once, CTAs a tile), at whole and ragged sizes, against 64 bits."""
import math
import random

import pytest
import torch

import gemm_affine_int4_gb300 as g4
from layer_ref import mm64, within

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def problem(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)

    def rows(n):   # (rows of different size)
        return torch.randn(n, K, generator=g, device="cuda") * (0.3 + torch.rand(n, 1, generator=g, device="cuda"))

    return g4.gai4_quantize_fp8(rows(N)) + g4.gai4_quantize_x_fp8(rows(M))


def check(M, N, K, dt):
    p = problem(M, N, K)
    out = g4.gai4_fp8_mm_t(*p, dtype=T[dt])
    assert g4.gai4_last_device_status() == 0
    within(out, *mm64(*p, T[dt]), f"mm {M} {N} {K}")
    assert torch.equal(out, g4.gai4_fp8_mm_t(*p, dtype=T[dt]))       # bit for bit


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(128, 4096, 4096), (127, 4097, 4112), (256, 4096, 4096), (100, 8000, 1024),
                                   (96, 5000, 8192), (250, 4100, 4000), (97, 7999, 1040)])
def test_128_tokens_at_once(M, N, K, dt):
    check(M, N, K, dt)


# (tokens and weight rows of a tile, CTAs that share one): sizes that take it on a GPU of 152 SMs, ragged in every direction
FORMS = {
    (16, 128, 1): [(9, 10004, 144), (35, 3472, 272)],
    (16, 128, 2): [(377, 155, 288), (22, 3066, 576)],
    (16, 128, 3): [(9, 151, 592), (35, 990, 1120)],
    (16, 128, 4): [(9, 154, 832), (50, 664, 1248)],
    (16, 128, 6): [(9, 151, 1440), (18, 643, 2224)],
    (16, 128, 8): [(9, 182, 1584), (17, 638, 2416)],
    (32, 128, 1): [(17, 10748, 144), (97, 2793, 272)],
    (32, 128, 2): [(17, 6146, 272), (73, 2055, 688)],
    (32, 128, 3): [(17, 2976, 656), (163, 790, 800)],
    (32, 128, 4): [(18, 2449, 864), (52, 1492, 1328)],
    (32, 128, 6): [(17, 1511, 1248), (33, 970, 3648)],
    (32, 128, 8): [(17, 1144, 1648), (69, 616, 2624)],
    (64, 128, 1): [(35, 10466, 144), (165, 3479, 272)],
    (64, 128, 2): [(35, 6937, 288), (99, 3307, 944)],
    (64, 128, 3): [(34, 3409, 608), (346, 841, 800)],
    (64, 128, 4): [(33, 3223, 832), (76, 2037, 1952)],
    (64, 128, 6): [(34, 2478, 1248), (117, 1288, 2880)],
    (64, 128, 8): [(38, 1586, 2352), (102, 803, 3648)],
    (128, 128, 1): [(65, 11954, 144), (114, 11101, 352)],
    (128, 128, 2): [(65, 6708, 320), (195, 3007, 1760)],
    (128, 128, 3): [(68, 4809, 944), (429, 1329, 1232)],
    (128, 128, 4): [(65, 4219, 832), (229, 1484, 2960)],
    (128, 128, 6): [(66, 2176, 2192), (370, 811, 4496)],
    (128, 128, 8): [(66, 1657, 2736), (241, 664, 5792)],
    (256, 192, 2): [(4992, 151, 320), (571, 2165, 528)],
    (256, 256, 2): [(271, 7897, 272), (535, 4829, 528)],
}


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes", [s for both in FORMS.values() for s in both])
def test_each_form(sizes, dt):
    check(*sizes, dt)


def test_every_form_that_is_taken_is_tested():
    """Where the SMs are divided otherwise, other sizes may take a form: the smallest that were found are checked here."""
    rng = random.Random(5)

    def upto(most):
        return int(round(math.exp(rng.uniform(0, math.log(most)))))

    taken = {}
    for _ in range(30000):
        sizes = upto(8192), upto(32768), 16 * upto(2048)
        form = g4.gai4_fp8_mm_t_plan(*sizes)
        assert form in FORMS
        if form not in taken or math.prod(sizes) < math.prod(taken[form]):
            taken[form] = sizes
    for form in set(taken) - {g4.gai4_fp8_mm_t_plan(*s) for both in FORMS.values() for s in both}:
        for dt in T:
            check(*taken[form], dt)
