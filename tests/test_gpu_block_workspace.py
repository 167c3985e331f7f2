"""GPU tests of workspaces of exactly the reported size, between canaries that must survive, and of the gradients of few bf16
rows with the weights in place and a ragged number of hidden columns."""
import pytest
import torch

from tests.block_reference import Ffn, Guarded, close, half_step
from tests.test_gpu_block import DT, PATHS, ffn_inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
FEW = [("bf16", 1, 64, 200), ("bf16", 7, 128, 200), ("bf16", 8, 1024, 1000), ("bf16", 9, 65, 4104), ("bf16", 16, 64, 1001),
       ("bf16", 17, 128, 333), ("f32", 1, 2048, 640), ("f32", 16, 5001, 40), ("f32", 17, 65, 9000), ("f32", 33, 1040, 513), ("f32", 64, 40, 5632)]


class Space:
    """A workspace of n bytes, 256-byte aligned, filled with 0xff, in a larger buffer."""
    EDGE = 4096

    def __init__(self, n, device):
        self.n, self.whole = n, torch.full((n + 2 * self.EDGE,), 0x5a, dtype=torch.uint8, device=device)
        self.t = self.whole[self.EDGE:self.EDGE + n]
        self.t.fill_(0xff)

    def check(self):
        torch.cuda.synchronize()
        assert (self.whole[:self.EDGE] == 0x5a).all() and (self.whole[self.EDGE + self.n:] == 0x5a).all(), "written outside"


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dt,rows,width,hidden", PATHS + FEW)
def test_feed_forward_stays_inside(cuda, dt, rows, width, hidden, bits):
    import rank_orthonormalized_optimizer_amd as dion
    t = DT[dt]
    X, scale, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, bits)

    def space(**kw):
        return Space(dion.gated_ffn_workspace_for(rows, width, hidden, cuda, t, x_dtype=X.dtype, **kw).numel(), cuda)
    gate, up = (torch.empty(rows, hidden, device=cuda, dtype=t) for _ in range(2))
    ws = space()
    Y = dion.gated_ffn_(X, Wg, Wu, Wd, scale=scale, gate=gate, up=up, workspace=ws.t)
    ws.check()
    assert torch.equal(Y, dion.gated_ffn_(X, Wg, Wu, Wd, scale=scale))
    for kept in ((gate, up), (None, None)):
        ws = space(for_grad=True, saved=kept[0] is not None)
        out, again = ([torch.empty_like(Y)] + [torch.empty_like(w) for w in (Wg, Wu, Wd)] for _ in range(2))
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, *kept, *out, scale=scale, workspace=ws.t)
        ws.check()
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, *kept, *again, scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("rows,width", [(2, 64), (70, 255), (5, 2050), (1300, 136), (2000, 4096), (300, 20001), (9, 65536)])
def test_norm_gradient_stays_inside(cuda, rows, width):
    import rank_orthonormalized_optimizer_amd as dion
    dY, h, w = (torch.randn(s, device=cuda) for s in ((rows, width), (rows, width), (width,)))
    rstd, dw, again = h.square().mean(1).rsqrt(), torch.empty_like(w), torch.empty_like(w)
    ws = Space(dion.rms_norm_grad_workspace_for(rows, width, cuda).numel(), cuda)
    dh, _ = dion.rms_norm_grad_(dY, h, w, rstd, dw, workspace=ws.t)
    ws.check()
    want, _ = dion.rms_norm_grad_(dY, h, w, rstd, again)
    assert torch.equal(dh, want) and torch.equal(dw, again)


@pytest.mark.parametrize("rows,width,hidden", [(1, 64, 200), (7, 128, 200), (8, 512, 1000), (16, 64, 1001), (17, 128, 333), (300, 192, 77)])
def test_gradients_in_place_over_a_ragged_reduction(cuda, rows, width, hidden):
    """width a multiple of 64, hidden none: dX's reduction over Wg's and Wu's rows in place, with one part or two of da and db."""
    import rank_orthonormalized_optimizer_amd as dion
    X, scale, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, "bf16", 16)
    out = {k: Guarded(v.shape, BF16, cuda) for k, v in (("dX", X), ("dWg", Wg), ("dWu", Wu), ("dWd", Wd))}
    dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, None, None, *(g.t for g in out.values()))
    want = Ffn(X, Wg, Wu, Wd, "silu", None, dY)
    for k, g in out.items():
        w, e = getattr(want, k), getattr(want, k + "_bound")
        close(g.check(), w, e + half_step(BF16) * (w.abs() + e), k)
