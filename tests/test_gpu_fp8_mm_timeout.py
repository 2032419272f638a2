"""The e4m3 product's way out of a wait that runs out: loads are withheld, the kernel takes back what it has in flight,
frees tensor memory and returns with GAI4_ERR_TIMEOUT, and the calls after it are as any others."""
import pytest
import torch

import gemm_affine_int4_gb300 as g4
from test_gpu_fp8_mm_forms import problem

pytestmark = pytest.mark.gpu
LIMIT = 1_000_000   # cycles a wait: half a millisecond

# pairs of CTAs: tiles of 192 weight rows, of 256, several tiles a pair
MANY = [(1500, 1700, 2048), (2304, 2048, 1040), (4096, 4096, 512)]


def give_up(shape, cases):
    p = problem(*shape)
    want = g4.gai4_fp8_mm_t(*p)
    out = torch.empty_like(want)
    for withheld, blocks in cases:
        assert g4.gai4_check_fp8_mm_wait(*p, out, withheld, blocks, LIMIT) == g4.GAI4_ERR_TIMEOUT
        # another kernel in the same shared and tensor memory
        assert torch.equal(g4.gai4_fp8_mm_t(*p), want)
    # the library's own status word was not touched; and what withholds nothing is the product
    assert g4.gai4_last_device_status() == 0
    for withheld, blocks in ((0, 0), (15, 1 << 20)):
        assert g4.gai4_check_fp8_mm_wait(*p, out.zero_(), withheld, blocks, 2_000_000_000) == 0
        assert torch.equal(out, want)


@pytest.mark.parametrize("withheld", [1, 2, 4, 8, 3, 12, 5, 10, 9, 6, 15])
@pytest.mark.parametrize("shape", MANY)
def test_pairs_of_ctas(shape, withheld):
    give_up(shape, [(withheld, blocks) for blocks in (0, 1, 3, 4, 6, 8)])


# few tokens: 16 to 128 at once, clusters of 1 to 8 CTAs; blocks that each CTA has at least
FEW = [((1, 4096, 4096), 8), ((64, 2048, 2048), 2), ((56, 5120, 17408), 17), ((128, 4096, 4096), 8), ((256, 4096, 4096), 8),
       ((16, 256, 16384), 16), ((40, 4096, 4096), 5), ((33, 300, 5136), 5), ((9, 20000, 2048), 2)]


@pytest.mark.parametrize("withheld", [3, 1, 2, 15])
@pytest.mark.parametrize("shape,least", FEW)
def test_few_tokens(shape, least, withheld):
    give_up(shape, [(withheld, blocks) for blocks in (0, 1, 2, 3, 4, 5, 6, 7, 12) if blocks < least])


@pytest.mark.parametrize("shape,least", FEW[:1] + FEW[2:4] + FEW[5:6])
def test_few_tokens_one_half_of_a_cluster(shape, least):
    """CTAs that have all of their loads beside CTAs that do not."""
    give_up(shape, [(withheld, blocks) for withheld in (4, 12, 3) for blocks in range(least)])
