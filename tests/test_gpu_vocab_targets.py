"""GPU tests of dW's target elements in bf16: D is rounded to bf16 for the products, and what that leaves of each target's
element is added to its row of dW in fp32, whatever the number of tokens, of rows, and of pieces of the vocabulary.

W = 0 makes every probability 1 / vocab exactly known and, with a vocabulary of 2^k, D's other elements g / vocab.  With g =
1 + 2^-8, the value furthest from its bf16 neighbours, a rounded D would leave 2^-8 of every target's element in the same
direction.  The others are off by at most 2^-8 g / vocab, together 2^-8 g n max|h| / vocab per element of dW, which a large
vocabulary makes small beside the output's own rounding."""
import math

import pytest
import torch

from tests.vocab_reference import U, half_step

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def expected(H, y, vocab, g):
    """dW for W = 0 in 64 bits, and the bound of its error: D's rounding away from the targets (2^-8 of g / vocab), the
    products' and the sums' additions (2 n u of the values added; the rest of a target's element is exact in fp32), the
    error of the probability (below 16 + 2 log(vocab) u of it; a target's element is 1 - p), and the output's rounding."""
    f64 = torch.float64
    keep = (y >= 0) & (y < vocab)
    h, t = H.to(f64)[keep], y[keep].long()
    gg = (g.to(f64).expand(y.numel()) if g.numel() == 1 else g.to(f64))[keep, None]
    p = 1.0 / vocab
    zero = torch.zeros(vocab, H.shape[1], dtype=f64, device=H.device)
    rows = zero.index_add(0, t, gg * h)
    size = zero.index_add(0, t, (gg * h).abs())
    all_ = (gg * h).sum(0, keepdim=True) * p
    every = (gg * h).abs().sum(0, keepdim=True) * p
    want = all_ - rows
    e = half_step(BF16) * (1 + 2.0 ** -7) * every + (2 * t.numel() + 16) * U * (every + size) \
        + (16 + 2 * math.log(vocab)) * U * (every + p * size)
    return want, e + half_step(BF16) * (want.abs() + e)


def check(dion, H, y, vocab, g, accumulate=False):
    dev = H.device
    W = torch.zeros(vocab, H.shape[1], dtype=BF16, device=dev)
    _, lse = dion.linear_cross_entropy_(H, W, y)
    ws = dion.linear_cross_entropy_workspace_for(y.numel(), vocab, H.shape[1], dev, BF16, for_grad=True).fill_(255)
    dW = torch.full_like(W, math.nan)
    dion.linear_cross_entropy_grad_(H, W, y, lse, g, None, dW, workspace=ws)
    want, bound = expected(H, y, vocab, g)
    off = (dW.double() - want).abs()
    assert not torch.isnan(off).any() and bool((off <= bound).all()), \
        f"{int((off > bound).sum())} of {off.numel()} elements over, worst {float((off / bound.clamp_min(1e-300)).max())} of the bound"
    again = torch.empty_like(dW)
    dion.linear_cross_entropy_grad_(H, W, y, lse, g, torch.empty_like(H), again)
    assert torch.equal(dW, again)


def inputs(device, tokens, vocab, width, key=0):
    gen = torch.Generator(device=device).manual_seed(tokens * 1000003 + vocab + width + key)
    u = torch.rand(tokens, generator=gen, device=device, dtype=torch.float64)
    y = (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1)
    H = (torch.randn(tokens, width, generator=gen, device=device) + 1).to(BF16)   # sums of one sign: no cancellation
    if tokens > 2:
        y[::7] = -100
        H[y == -100] = math.nan
    return H, y


# one to sixteen tokens (a kernel of their own), up to 128, more; sliced products; sorted by counting and by radix; rows of
# any length; fewer tokens than rows of a piece, and more
@pytest.mark.parametrize("tokens,vocab,width", [(1, 4096, 8), (2, 4096, 64), (8, 8192, 72), (16, 4096, 255), (17, 4096, 8),
                                                (33, 8192, 64), (100, 4096, 1001), (129, 16384, 36), (300, 4096, 2100),
                                                (700, 65536, 128), (4097, 65536, 66), (16385, 65536, 24), (20000, 32768, 64)])
@pytest.mark.parametrize("per_token", [False, True])
def test_frequent_targets(cuda, tokens, vocab, width, per_token):
    import rank_orthonormalized_optimizer_amd as dion
    H, y = inputs(cuda, tokens, vocab, width)
    g = torch.full((tokens if per_token else 1,), 1 + 2.0 ** -8, device=cuda)
    print(f"[targets] {tokens} x {vocab} x {width}", flush=True)
    check(dion, H, y, vocab, g)


@pytest.mark.parametrize("tokens,vocab,width", [(65536, 16384, 32), (40000, 16384, 24), (200001, 8192, 16), (300, 1 << 21, 8)])
def test_targets_in_pieces_of_the_vocabulary(cuda, tokens, vocab, width):
    """Rows summed per row of the piece (many tokens) or per token (few); targets of one id, of ids at the pieces' borders."""
    import rank_orthonormalized_optimizer_amd as dion
    H, y = inputs(cuda, tokens, vocab, width)
    g = torch.full((tokens,), 1 + 2.0 ** -8, device=cuda)
    print(f"[targets] {tokens} x {vocab} x {width}", flush=True)
    check(dion, H, y, vocab, g)
    H = torch.where(torch.isnan(H), 1.0, H)   # no target is ignored from here on
    check(dion, H, torch.full_like(y, vocab - 1), vocab, g)
    edge = torch.arange(tokens, device=cuda) % 3 - 1 + vocab // 2   # the two sides of the middle
    check(dion, H, edge, vocab, g)


@pytest.mark.parametrize("accumulate", [False, True])
def test_no_target_counts(cuda, accumulate):
    """Every target ignored: no row gets anything, whatever the last call left in the workspace."""
    import rank_orthonormalized_optimizer_amd as dion
    H, y = inputs(cuda, 300, 4096, 64)
    W = torch.zeros(4096, 64, dtype=BF16, device=cuda)
    g = torch.full((300,), 1 + 2.0 ** -8, device=cuda)
    ws = dion.linear_cross_entropy_workspace_for(300, 4096, 64, cuda, BF16, for_grad=True)
    dW = torch.zeros_like(W)
    _, lse = dion.linear_cross_entropy_(H, W, y)
    dion.linear_cross_entropy_grad_(H, W, y, lse, g, None, dW, workspace=ws)
    assert dW.any()
    none = torch.full_like(y, -100)
    dW.fill_(3 if accumulate else math.nan)
    dion.linear_cross_entropy_grad_(H, W, none, lse, g, None, dW, accumulate=accumulate, workspace=ws)
    assert (dW == (3 if accumulate else 0)).all()
