"""The example's decoder layer runs, positions go on from step to step, and a token's output does not depend on the
requests beside it."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_runs(capsys):
    import fp8_decoder_layer as ex
    layer = ex.main()
    assert layer.lens.tolist() == [309, 203, 129]
    assert int(layer.free_count) == 24 - 10 - 7 - 5


def test_positions_go_on():
    import fp8_decoder_layer as ex
    layer = ex.Layer(2, 160, 10, seed=4)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(80, ex.HIDDEN, generator=torch.Generator().manual_seed(3)).to(ex.T).cuda()
    _, plan = layer.step(x, ints(30, 50), 50)
    assert plan.positions.tolist() == list(range(30)) + list(range(50))
    y, plan = layer.step(x[:3], ints(2, 1), 2)
    assert plan.positions.tolist() == [30, 31, 50] and y.shape == (3, ex.HIDDEN) and bool(y.isfinite().all())


def test_a_request_alone_and_beside_another():
    """The same tokens of one request with another request's in front or without: products of 20 and of 25 rows take the
    same number of tokens at once and parts of K, attention the same few-row kernel, so rows are equal bit for bit."""
    import fp8_decoder_layer as ex
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(25, ex.HIDDEN, generator=torch.Generator().manual_seed(5)).to(ex.T).cuda()
    alone, both = ex.Layer(1, 64, 4, seed=6), ex.Layer(2, 64, 4, seed=6)
    y, _ = alone.step(x[5:], ints(20), 0)
    z, _ = both.step(x, ints(5, 20), 0)
    assert torch.equal(y, z[5:])
