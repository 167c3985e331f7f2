"""GPU tests of the rounding of the stream that the norm to 8 bits writes."""
import pytest
import torch

from tests.block_reference import F64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


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


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(70, 255), (33, 1024), (9, 1500), (3, 2048), (7, 2050), (3, 5001), (2, 20001)])
def test_the_stream_is_the_sum_rounded_once(cuda, rows, width, t):
    """Without dropout the sum is exact in 64 bits, but for numbers further apart than its 53."""
    import rank_orthonormalized_optimizer_amd as dion
    g = torch.Generator(device=cuda).manual_seed(width)
    x, r = (torch.randn(rows, width, generator=g, device=cuda) for _ in range(2))
    r = r.to(t)
    exact = x.to(F64) + r.to(F64)
    if t == F32:
        want = exact.float().to(F64)
    else:   # to nearest, ties to even, as torch.round has them
        step = torch.exp2(torch.floor(torch.log2(exact.abs())) - 7)
        want = torch.round(exact / step) * step
    _, _, h, _ = dion.rms_norm_8bit_(x, torch.ones(width, device=cuda), residual=r)
    assert torch.equal(h.to(F64), want)
