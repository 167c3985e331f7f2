"""Calls of MixedDion that gather gradients run on the current stream, where ``step`` reads them: none takes another (no GPU
needed)."""
import inspect

import pytest
import torch

import rank_orthonormalized_optimizer_amd as dion

GATHER = ("lookup_grad", "head_loss", "norm_grad", "feed_forward_grad")


@pytest.mark.parametrize("name", GATHER)
def test_no_stream_among_the_arguments(name):
    kinds = {p.name: p.kind for p in inspect.signature(getattr(dion.MixedDion, name)).parameters.values()}
    assert "stream" not in kinds and inspect.Parameter.VAR_KEYWORD not in kinds.values()


def test_norm_grad_refuses_a_stream():
    opt = dion.MixedDion([torch.ones(8)])
    x, rstd = torch.zeros(3, 8), torch.ones(3)
    with pytest.raises(TypeError, match="stream"):
        opt.norm_grad(0, x, x, rstd, stream=None)
    assert not opt.gathered and not opt.pending
    with pytest.raises(ValueError, match="GPU"):   # its other arguments reach the call
        opt.norm_grad(0, x, x, rstd, dsum=x, p=0.1, seed=None, site=3, dh=x, dx=x)
