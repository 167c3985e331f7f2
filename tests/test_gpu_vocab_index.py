"""GPU tests of how MixedDion's vocabulary calls name a parameter: from the back as from the front, and none that is not there."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_parameters_named_from_the_back(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    gen = torch.Generator(device=cuda).manual_seed(6)
    params = [torch.randn(32, 32, generator=gen, device=cuda), torch.randn(50, 32, generator=gen, device=cuda)]
    a, b = (dion.MixedDion([p.clone() for p in params]) for _ in range(2))
    ids = torch.randint(0, 50, (64,), generator=gen, device=cuda)
    dY = torch.randn(64, 32, generator=gen, device=cuda)
    other = torch.randn(32, 32, generator=gen, device=cuda)
    assert torch.equal(a.lookup(-1, ids), b.lookup(1, ids))
    a.lookup_grad(-1, ids, dY)
    a.lookup_grad(np.int64(1), ids, dY)          # the same parameter: adds up
    a.head_loss(-1, dY, ids)
    for _ in range(2):
        b.lookup_grad(1, ids, dY)
    b.head_loss(1, dY, ids)
    assert torch.equal(a.gathered[1], b.gathered[1])
    a.step([other, None])
    b.step([other, None])
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))


@pytest.mark.parametrize("i,error", [(2, IndexError), (-3, IndexError), (1.0, TypeError), ("1", TypeError)])
def test_parameters_that_are_not_there(cuda, i, error):
    import rank_orthonormalized_optimizer_amd as dion
    opt = dion.MixedDion([torch.zeros(8, 8, device=cuda), torch.zeros(9, 8, device=cuda)])
    ids, rows = torch.zeros(3, dtype=torch.int64, device=cuda), torch.zeros(3, 8, device=cuda)
    for call in (lambda: opt.lookup(i, ids), lambda: opt.lookup_grad(i, ids, rows), lambda: opt.head_loss(i, rows, ids)):
        with pytest.raises(error):
            call()
    assert not opt.gathered and not opt.pending
