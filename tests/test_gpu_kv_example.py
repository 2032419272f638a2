"""The example's layer runs, and gives what the same layer gives when every step reads the whole sequence anew."""
import os
import sys

import pytest
import torch

import gemm_affine_int4_gb300 as g4

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_runs(capsys):
    import paged_attention_layer as ex
    layer = ex.main()
    assert layer.lens.tolist() == [309, 203, 129]
    assert int(layer.free_count) == 24 - 10 - 7 - 5


def test_steps_equal_one_long_step():
    """A prompt in one step against the same tokens in several (last token's output): the cached rows are the same, so
    the outputs differ by the kernels' rounding only: one bf16 spacing of keys, values and probabilities (3 * 2^-8 of
    sum p |v|, below the largest |v|) before the output projection, whose rows have a sum of squares near 1."""
    import paged_attention_layer as ex
    x = torch.randn(150, ex.HIDDEN, generator=torch.Generator().manual_seed(3)).to(ex.T).cuda()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    one, many = ex.Layer(1, 160, 5, seed=4), ex.Layer(1, 160, 5, seed=4)
    y, plan = one.step(x, ints(150), 150)
    at = 0
    for n in (100, 30, 4, 1, 14, 1):
        z, p = many.step(x[at:at + n], ints(n), n)
        at += n
    assert torch.equal(one.table, many.table) and one.lens.tolist() == many.lens.tolist() == [150]
    rows = [g4.gai4_kv_read(c, plan.slots, group_size=ex.GROUP) for c in (one.k_cache, many.k_cache)]
    # the projections of one row and of many round weights differently: codes may differ where a value lies between two
    assert float((rows[0] - rows[1]).norm() / rows[0].norm()) < 0.02
    assert float((y[-1].float() - z[-1].float()).norm() / y[-1].float().norm()) < 0.05
