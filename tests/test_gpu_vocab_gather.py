"""GPU tests of the gradients that MixedDion gathers for its vocabulary matrices: contributions of any type add up in fp32."""
import math

import pytest
import torch

from tests.vocab_reference import Head, table

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dt", [F32, BF16])
def test_small_contributions_are_kept(cuda, dt):
    """One contribution of 1 and 300 of 2^-12 to the same rows: sums of powers of two, exact in fp32, lost in bf16."""
    import rank_orthonormalized_optimizer_amd as dion
    opt = dion.MixedDion([torch.zeros(40, 24, dtype=dt, device=cuda)])
    ids = torch.arange(30, device=cuda)
    opt.lookup_grad(0, ids, torch.ones(30, 24, dtype=dt, device=cuda))
    for _ in range(300):
        opt.lookup_grad(0, ids, torch.full((30, 24), 2.0 ** -12, dtype=dt, device=cuda))
    got = opt.gathered[0].double()
    assert (got[:30] == 1 + 300 * 2.0 ** -12).all() and (got[30:] == 0).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab,width", [(12, 70, 24), (48, 300, 64), (300, 1000, 72)])
def test_tied_microbatches(cuda, tokens, vocab, width, dt):
    """Eight microbatches of head and table against 64 bits: each call within its bound of the sums before it."""
    import rank_orthonormalized_optimizer_amd as dion
    gen = torch.Generator(device=cuda).manual_seed(tokens)
    W = (torch.randn(vocab, width, generator=gen, device=cuda) / 8).to(dt)
    opt = dion.MixedDion([W])
    want = torch.zeros(vocab, width, dtype=torch.float64, device=cuda)
    bound = torch.zeros_like(want)
    print(f"[gather] {tokens} x {vocab} x {width} {dt}", flush=True)
    for k in range(8):
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device=cuda)
        y = torch.where(ids % 5 == 0, -100, (ids * 7 + 3) % vocab)
        H = torch.randn(tokens, width, generator=gen, device=cuda).to(dt)
        grad = torch.rand(tokens, generator=gen, device=cuda) if k % 2 else None
        _, dH = opt.head_loss(0, H, y, grad)
        used = grad if grad is not None else torch.full((1,), 1.0, device=cuda) / (y != -100).sum()
        head = Head(H, W, y, grad=used, dw_dtype=F32, dw_old=want)
        want, bound = head.dW, bound * (1 + 2.0 ** -22) + head.dW_bound
        dY = torch.randn(tokens, width, generator=gen, device=cuda).to(dt)
        opt.lookup_grad(0, ids, dY, 3.0)
        want, e = table(ids, dY, vocab, 3.0, old=want)
        bound = bound * (1 + 2.0 ** -22) + e + 2.0 ** -24 * want.abs()
    off = (opt.gathered[0].double() - want).abs()
    assert opt.gathered[0].dtype == F32 and bool((off <= bound).all()), float((off / bound).max())
    # and that bound is far below a bf16 rounding of the sums
    assert float(bound.norm()) <= 2.0 ** -12 * float(want.norm())


def test_step_takes_gathered_beside_given_gradients(cuda):
    """Two bf16 matrices of one shape, a stack: one gradient gathered in fp32, one given in bf16."""
    import rank_orthonormalized_optimizer_amd as dion
    gen = torch.Generator(device=cuda).manual_seed(1)
    params = [(torch.randn(90, 64, generator=gen, device=cuda) / 8).to(BF16) for _ in range(2)]
    a = dion.MixedDion([p.clone() for p in params])
    b = dion.MixedDion([p.clone() for p in params])
    ids = torch.randint(0, 90, (500,), generator=gen, device=cuda)
    dY = torch.randn(500, 64, generator=gen, device=cuda).to(BF16)
    other = torch.randn(90, 64, generator=gen, device=cuda).to(BF16)
    for _ in range(2):
        a.lookup_grad(0, ids, dY, math.sqrt(64))
        gathered = a.gathered[0].clone()
        a.step([None, other])
        b.step([gathered, other.float()])
        torch.cuda.synchronize()
        for p, q in zip(a.params, b.params):
            assert p.dtype == BF16 and torch.equal(p, q)
