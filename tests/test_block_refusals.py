"""Every tensor that a forward call of the residual blocks reads or fills is refused where it requires a gradient and autograd
records (no GPU needed)."""
import pytest
import torch

import rank_orthonormalized_optimizer_amd as dion


def tensors():
    x, W = torch.zeros(3, 8), torch.zeros(16, 8)
    rows, inner = torch.zeros(3), torch.zeros(3, 16)
    norm = dict(x=x, w=torch.zeros(8), residual=x.clone(), h=x.clone(), out=x.clone(), rstd=rows)
    return {"dropout_": dict(x=x, p=0.1, residual=x.clone(), out=x.clone()), "rms_norm_": norm,
            "rms_norm_8bit_": dict(norm, scale=rows.clone()),
            "gated_ffn_": dict(X=x, Wg=W, Wu=W.clone(), Wd=W.t().contiguous(), scale=rows, gate=inner, up=inner.clone(), out=x.clone())}


CASES = [(call, name) for call, kw in tensors().items() for name, t in kw.items() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("call,name", CASES)
def test_refused(call, name):
    kw = tensors()[call]
    kw[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        getattr(dion, call)(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):   # taken, up to the next check
        getattr(dion, call)(**kw)
