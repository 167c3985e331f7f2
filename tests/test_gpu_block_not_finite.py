"""GPU tests of what the feed-forward block's gradients make of numbers that are not finite."""
import pytest
import torch

from tests.test_gpu_block import DT, PATHS, ffn_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt,rows,width,hidden", PATHS)
def test_a_nan_reaches_every_gradient_of_its_column(cuda, dt, rows, width, hidden, act):
    """A NaN in one row of Wg makes a's column NaN, so da and db of that column, kept or formed again: its rows of dWg and dWu and
    all of dX."""
    import rank_orthonormalized_optimizer_amd as dion
    t, at = DT[dt], hidden - 1
    X, _, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, 16)
    Wg[at, width // 2] = float("nan")
    gate, up = (torch.empty(rows, hidden, device=cuda, dtype=t) for _ in range(2))
    Y = dion.gated_ffn_(X, Wg, Wu, Wd, act=act, gate=gate, up=up)
    assert torch.isnan(Y).all()
    for kept in ((gate, up), (None, None)):
        dX, dWg, dWu, dWd = out = [torch.empty_like(v) for v in (X, Wg, Wu, Wd)]
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, *kept, *out, act=act)
        assert torch.isnan(dX).all()
        for name, g, rest in (("dWg", dWg[at], dWg[:at]), ("dWu", dWu[at], dWu[:at]), ("dWd", dWd[:, at], dWd[:, :at])):
            assert torch.isnan(g).all(), name
            assert torch.isfinite(rest).all(), name


@pytest.mark.parametrize("dt,rows,width,hidden", PATHS)
def test_an_infinite_weight_of_the_second_product_reaches_its_column_alone(cuda, dt, rows, width, hidden):
    """du's other columns, and so the other rows of dWg and dWu, stay as they were, bit for bit."""
    import rank_orthonormalized_optimizer_amd as dion
    X, _, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, 16)
    Wd[width // 2, 1] = 0

    def run():
        dWg, dWu = torch.empty_like(Wg), torch.empty_like(Wu)
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, None, None, None, dWg, dWu)
        return dWg, dWu
    clean = run()
    Wd[width // 2, 1] = float("inf")
    rest = torch.arange(hidden, device=cuda) != 1
    for a, b in zip(run(), clean):
        assert not torch.isfinite(a[1]).any() and torch.equal(a[rest], b[rest])
