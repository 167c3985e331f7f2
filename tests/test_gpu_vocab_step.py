"""GPU tests of MixedDion.step's refusals: a refused step changes nothing and keeps the gathered gradients."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def setup(device):
    import rank_orthonormalized_optimizer_amd as dion
    gen = torch.Generator(device=device).manual_seed(4)
    params = [(torch.randn(*s, generator=gen, device=device) / 8) for s in ((50, 32), (32, 32), (32,), (50, 32))]
    a = dion.MixedDion([p.clone() for p in params])
    b = dion.MixedDion([p.clone() for p in params])
    ids = torch.randint(0, 50, (100,), generator=gen, device=device)
    dY = torch.randn(100, 32, generator=gen, device=device)
    given = [torch.randn(*p.shape, generator=gen, device=device) for p in params]
    return a, b, ids, dY, given


@pytest.mark.parametrize("kind,error", [("short", ValueError), ("missing", ValueError), ("both", ValueError),
                                        ("shape", ValueError), ("bias", ValueError), ("dtype", TypeError),
                                        ("host", ValueError), ("number", TypeError)])
def test_refused_step_keeps_what_was_gathered(cuda, kind, error):
    a, b, ids, dY, given = setup(cuda)
    for opt in (a, b):
        opt.lookup_grad(0, ids, dY, 2.0)
    before = [p.clone() for p in a.params]
    bad = [None] + given[1:]
    if kind == "short":
        bad = bad[:3]
    elif kind == "missing":
        bad[1] = None
    elif kind == "both":
        bad[0] = given[0]
    elif kind == "shape":
        bad[3] = given[3].t().contiguous()
    elif kind == "bias":
        bad[2] = given[2][:31]
    elif kind == "dtype":
        bad[1] = given[1].double()
    elif kind == "host":
        bad[1] = given[1].cpu()
    else:
        bad[1] = 1.0
    with pytest.raises(error):
        a.step(bad)
    assert a.t == 0 and all(torch.equal(p, q) for p, q in zip(a.params, before))
    for opt in (a, b):   # the next microbatch adds to the first
        opt.lookup_grad(0, ids, dY, 1.0)
        opt.step([None] + given[1:])
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
    with pytest.raises(ValueError, match="no gradient"):
        a.step([None] + given[1:])


def test_more_gradients_than_parameters_are_not_looked_at(cuda):
    a, b, _, _, given = setup(cuda)
    a.step(given + [None, "more"])
    b.step(given)
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
