"""Calls without rows, whose arrays of rows may be NULL as empty tensors are (no GPU needed but for the last)."""
import pytest
import torch

from rank_orthonormalized_optimizer_amd import _lib
from tests.test_block_abi import ffn_grad

EMPTY = dict(rows=0, X=0, dY=0, gate=0, up=0, dX=0, ws=0)


def test_the_input_s_gradient_alone():
    assert ffn_grad(**EMPTY, dWg=0, dWu=0, dWd=0) == _lib.OK
    assert ffn_grad(**EMPTY, dWg=0, dWu=0, dWd=0, acc=1) == _lib.OK
    assert ffn_grad(**EMPTY, acc=1) == _lib.OK


def test_still_refused():
    assert ffn_grad(**EMPTY, dWg=0, dWd=0) == _lib.ERR_NULL
    assert ffn_grad(rows=1, dX=0, dWg=0, dWu=0, dWd=0) == _lib.ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_empty_tensors(cuda, t):
    import rank_orthonormalized_optimizer_amd as dion
    X, Wg, Wu, Wd = (torch.randn(s, device=cuda).to(t) for s in ((2, 0, 24), (40, 24), (40, 24), (24, 40)))
    gate = torch.empty(2, 0, 40, device=cuda, dtype=t)
    for kept in ((None, None), (gate, gate.clone())):
        dX = torch.empty_like(X)
        assert dion.gated_ffn_grad_(X, Wg, Wu, Wd, X, *kept, dX)[0] is dX
    opt = dion.MixedDion([Wg, Wu, Wd])
    assert opt.feed_forward_grad((0, 1, 2), X, X, opt.feed_forward((0, 1, 2), X)[1]).shape == X.shape
    assert all((opt.gathered[i] == 0).all() for i in range(3))
