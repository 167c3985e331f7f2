"""GPU tests of the norm where the squares of a row leave fp32's range, and of the rounding of the stream that it writes."""
import pytest
import torch

from tests.block_reference import F64, Norm, close, half_step

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


def test_the_stream_of_the_8_bit_norm_is_rounded_once(cuda):
    """Sums just above and below the middle between two bf16 numbers, by less than fp32 can tell: to fp32 first they would be the
    middle, which goes to the even one."""
    import rank_orthonormalized_optimizer_amd as dion
    width = 256
    r = torch.randint(128, 256, (9, width), device=cuda, generator=torch.Generator(device=cuda).manual_seed(1)).to(F32) / 128
    r = r.to(BF16)   # [1, 2), steps of 2^-7
    r[1::2] *= -1
    tiny = 2.0 ** -30
    x = torch.full((9, width), 2.0 ** -8, device=cuda)   # half a step, which 2^-30 more or less decides
    x = torch.where(torch.arange(width, device=cuda) % 2 == 0, x + tiny, x - tiny)
    x[::3] *= -1
    exact = x.to(F64) + r.to(F64)
    step = torch.exp2(torch.floor(torch.log2(exact.abs())) - 7)
    want = torch.round(exact / step) * step   # (no ties)
    _, _, h, _ = dion.rms_norm_8bit_(x, torch.ones(width, device=cuda), residual=r)
    assert h.dtype == BF16 and torch.equal(h.to(F64), want)
