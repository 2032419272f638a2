"""The e4m3 product in each of its forms (tokens at once, CTAs a tile), at whole and ragged sizes, against 64 bits."""
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
