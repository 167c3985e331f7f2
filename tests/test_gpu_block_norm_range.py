"""GPU tests of the norm where the squares of a row leave fp32's range."""
import pytest
import torch

from tests.block_reference import Norm, close, half_step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("width", [1, 7, 513, 2050, 8200, 20001])
def test_rows_whose_squares_leave_the_range(cuda, width, t):
    """Finite rows far from 1, with eps 0: their squares overflow or underflow fp32, the norm does not."""
    import rank_orthonormalized_optimizer_amd as dion
    g = torch.Generator(device=cuda).manual_seed(width)
    sizes = torch.tensor([1.0, 1e25, 1e37, 2.0 ** 64, 1e-25, 1e-33, 2.0 ** -64, 3e18], device=cuda)
    x = (torch.randn(sizes.numel(), width, generator=g, device=cuda).clamp(-5, 5) * sizes[:, None]).to(t)
    w = torch.randn(width, generator=g, device=cuda).to(t)
    y, _, rstd = dion.rms_norm_(x, w, 0.0)
    want = Norm(x, w, 0.0)
    close(rstd, want.rstd, want.rstd_bound, "rstd")
    close(y, want.y, want.y_bound + half_step(t) * (want.y.abs() + want.y_bound), "y")
    y, _, rstd = dion.rms_norm_(x, w, 1e-6)   # where eps is larger than the small rows
    want = Norm(x, w, 1e-6)
    close(rstd, want.rstd, want.rstd_bound, "rstd")
    close(y, want.y, want.y_bound + half_step(t) * (want.y.abs() + want.y_bound) + 2.0 ** -149, "y")


def test_rows_of_zeros_and_not_finite_ones_beside_the_range(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    x, w = torch.zeros(4, 300, device=cuda), torch.ones(300, device=cuda)
    x[1, 3], x[2, 3], x[3] = float("inf"), float("nan"), 1e30
    for eps in (0.0, 1e-30, 1e-6):
        y, _, rstd = dion.rms_norm_(x, w, eps)
        assert torch.isnan(y[0]).all() if eps == 0 else (y[0] == 0).all()   # 0 / 0
        assert torch.isnan(y[1, 3]) and (y[1, :3] == 0).all() and torch.isnan(y[2]).all()
        assert ((y[3] - 1).abs() <= 2.0 ** -22).all()
