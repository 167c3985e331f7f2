"""GPU tests of batches whose mask leaves no target: the factor of a mean over the targets that count is 1 / 0 then, and
must reach neither dH nor dW."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# dW by rows (up to 16 tokens), in few, small and large tiles, with sliced products, beside sums per target
@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,vocab,width", [(1, 50, 40), (9, 50, 40), (20, 50, 40), (300, 50, 40), (2048, 300, 1030),
                                                (20000, 3000, 264)])
@pytest.mark.parametrize("factor", [math.inf, -math.inf, math.nan])
def test_factor_without_targets(cuda, tokens, vocab, width, dt, wdt, factor):
    import rank_orthonormalized_optimizer_amd as dion
    gen = torch.Generator(device=cuda).manual_seed(tokens)
    H = torch.randn(tokens, width, generator=gen, device=cuda).to(DT[dt])
    W = torch.randn(vocab, width, generator=gen, device=cuda).to(DT[dt])
    none = torch.full((tokens,), -100, device=cuda)
    loss, lse = dion.linear_cross_entropy_(H, W, none)
    old = torch.randn(vocab, width, generator=gen, device=cuda).to(DT[wdt])
    print(f"[no targets] {tokens} x {vocab} x {width} {dt} {wdt}", flush=True)
    for g in (torch.full((1,), factor, device=cuda), torch.full((tokens,), factor, device=cuda)):
        dH, dW = torch.full_like(H, 3), old.clone()
        dion.linear_cross_entropy_grad_(H, W, none, lse, g, dH, dW, accumulate=True)
        assert not dH.any() and torch.equal(dW, old)
        dion.linear_cross_entropy_grad_(H, W, none, lse, g, dH, dW)
        assert not dH.any() and not dW.any()
        dW.copy_(old)
        dion.linear_cross_entropy_grad_(H, W, none, lse, g, None, dW, accumulate=True)
        assert torch.equal(dW, old)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_factor_reaches_the_tokens_that_count(cuda, dt):
    """One counted token of many: an infinite factor is its own, as the formula has it."""
    import rank_orthonormalized_optimizer_amd as dion
    gen = torch.Generator(device=cuda).manual_seed(3)
    H = torch.randn(300, 40, generator=gen, device=cuda).to(DT[dt])
    W = torch.randn(50, 40, generator=gen, device=cuda).to(DT[dt])
    y = torch.full((300,), -100, device=cuda)
    y[7] = 3
    _, lse = dion.linear_cross_entropy_(H, W, y)
    dH, dW = torch.empty_like(H), torch.empty_like(W)
    dion.linear_cross_entropy_grad_(H, W, y, lse, torch.full((1,), math.inf, device=cuda), dH, dW)
    assert not torch.isfinite(dH[7].float()).any() and not torch.isfinite(dW.float()).any()
    dH[7] = 0
    assert not dH.any()
