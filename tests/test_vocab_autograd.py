"""The vocabulary operators record no graph: they refuse tensors that require a gradient where one would be recorded, and
take them where none would, so that no parameter silently stays without its gradient."""
import pytest
import torch

import rank_orthonormalized_optimizer_amd as dion


def tensors(device, which):
    t = {"W": torch.ones(10, 16, device=device), "H": torch.ones(4, 16, device=device)}
    t[which].requires_grad_()
    return t["W"], t["H"], torch.zeros(4, dtype=torch.int64, device=device)


@pytest.mark.parametrize("which", ["W", "H"])
def test_refused_without_a_gpu(which):
    W, H, ids = tensors("cpu", which)
    with pytest.raises(ValueError, match=f"{which} requires a gradient"):
        dion.linear_cross_entropy_(H, W, ids)
    if which == "W":
        with pytest.raises(ValueError, match="W requires a gradient.*embedding_grad_"):
            dion.embedding_(ids, W)
    else:
        with pytest.raises(ValueError, match="GPU"):   # no gradient asked for: the next check speaks
            dion.embedding_(ids, W)


def test_written_tensors_refused():
    W, H, ids = torch.ones(10, 16), torch.ones(4, 16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="out requires a gradient"):
        dion.embedding_(ids, W, out=torch.zeros(4, 16, requires_grad=True))
    with pytest.raises(ValueError, match="loss requires a gradient"):
        dion.linear_cross_entropy_(H, W, ids, loss=torch.zeros(4, requires_grad=True))


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["W", "H"])
def test_taken_where_no_graph_is_recorded(cuda, which):
    W, H, ids = tensors(cuda, which)
    with torch.no_grad():
        y, (loss, lse) = dion.embedding_(ids, W), dion.linear_cross_entropy_(H, W, ids)
    assert torch.equal(y, dion.embedding_(ids, W.detach()))
    assert torch.equal(loss, dion.linear_cross_entropy_(H.detach(), W.detach(), ids)[0])
    # the gradients are asked for outright: their tensors may require one
    dH, dW = torch.empty_like(H, requires_grad=False), torch.empty_like(W, requires_grad=False)
    dion.linear_cross_entropy_grad_(H, W, ids, lse, torch.ones(1, device=cuda), dH, dW)
    dion.embedding_grad_(ids, dH, dW, accumulate=True)
    # and MixedDion's calls are a training loop's own
    opt = dion.MixedDion([W])
    opt.lookup(0, ids)
    loss2, dH2 = opt.head_loss(0, H, ids, torch.ones(1, device=cuda))
    assert torch.equal(loss2, loss) and torch.equal(dH2, dH)
