"""GPU tests of the vocabulary operators (lookup, table gradient, linear cross entropy and its
gradients) against their definitions in 64 bits, at the sizes and masks where they can go wrong.
Every output lies between canaries that must survive, and every workspace starts out filled with
NaN bit patterns."""
import math

import pytest
import torch

from tests.vocab_reference import Head, half_step, table

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF16}
CANARY = 64   # elements on either side


class Guarded:
    """A tensor inside a larger buffer whose borders hold a pattern."""

    def __init__(self, shape, dtype, device, fill=math.nan):
        n = math.prod(shape)
        self.whole = torch.full((n + 2 * CANARY + 16,), 1234.0, dtype=dtype, device=device)
        self.t = self.whole[CANARY:CANARY + n].view(shape)
        self.t.fill_(fill)
        self.n = n

    def check(self):
        torch.cuda.synchronize()
        assert (self.whole[:CANARY] == 1234.0).all() and (self.whole[CANARY + self.n:] == 1234.0).all()
        return self.t


def dirty(ws):
    return ws.fill_(255)


def gen(device, *key):
    seed = 17
    for k in key:
        seed = seed * 1000003 + int(k)
    return torch.Generator(device=device).manual_seed(seed % (1 << 62))


def skewed_ids(g, n, vocab, device, dtype=torch.int64):
    u = torch.rand(n, generator=g, device=device, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1).to(dtype)


def close(got, want, bound, what):
    got = got.to(torch.float64).reshape(want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN where none belongs, or none where one does"
    fine = ~torch.isnan(want)
    worst = ((got - want).abs() - bound)[fine]
    assert worst.numel() == 0 or float(worst.max()) <= 0, \
        f"{what}: {float((got - want).abs()[fine].max())} off, {int((worst > 0).sum())} values over their bound"


# ---------------------------------------------------------------------------- lookup
@pytest.mark.parametrize("wdt,odt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,vocab,width", [(0, 5, 8), (1, 1, 1), (3, 7, 5), (65, 33, 12), (1, 1000, 2048), (513, 129, 64),
                                                (70, 31, 4104), (1030, 50, 255)])
def test_lookup(cuda, tokens, vocab, width, wdt, odt):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, vocab, width)
    W = torch.randn(vocab, width, generator=g, device=cuda).to(DT[wdt])
    for idt in (torch.int32, torch.int64):
        ids = torch.randint(0, vocab, (tokens,), generator=g, device=cuda).to(idt)
        scale = 1.7
        out = Guarded((tokens, width), DT[odt], cuda)
        assert dion.embedding_(ids, W, scale, out.t) is out.t
        want = (W[ids.long()].float() * torch.tensor(scale, dtype=F32, device=cuda)).to(DT[odt])
        assert torch.equal(out.check(), want)


def test_lookup_shapes_and_bad_ids(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    W = torch.randn(10, 24, device=cuda, dtype=BF16)
    ids = torch.tensor([[0, 9, -1], [10, 3, 1 << 40]], device=cuda)
    out = dion.embedding_(ids, W)
    assert out.shape == (2, 3, 24) and out.dtype == BF16
    bad = (ids < 0) | (ids >= 10)
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], W[ids[~bad]])


# ---------------------------------------------------------------------------- table gradient
TABLE = [(0, 5, 8), (1, 1, 1), (1, 300, 64), (2, 3, 3), (15, 4, 12), (16, 4, 8), (17, 4, 8), (64, 1, 255), (1000, 40, 36),
         (1025, 70000, 8), (4097, 300, 24), (5000, 257, 40), (16384, 1000, 8), (16385, 1000, 8), (40000, 66000, 4),
         (33000, 3, 16), (300, 1 << 17, 5), (777, 100, 1040), (600, 50, 2049)]


@pytest.mark.parametrize("ydt,wdt,accumulate", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "f32", True),
                                                ("f32", "bf16", True)])
@pytest.mark.parametrize("tokens,vocab,width", TABLE)
def test_table_gradient(cuda, tokens, vocab, width, ydt, wdt, accumulate):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, vocab, width)
    ids = skewed_ids(g, tokens, vocab, cuda, torch.int32 if tokens % 2 else torch.int64)
    dY = torch.randn(tokens, width, generator=g, device=cuda).to(DT[ydt])
    dW = Guarded((vocab, width), DT[wdt], cuda)
    dW.t.copy_(torch.randn(vocab, width, generator=g, device=cuda))
    old = dW.t.clone() if accumulate else None
    pad = 2 if vocab > 2 else -1
    scale = 0.75
    ws = dirty(dion.embedding_grad_workspace_for(tokens, vocab, width, cuda))
    assert dion.embedding_grad_(ids, dY, dW.t, scale, padding_id=pad, accumulate=accumulate, workspace=ws) is dW.t
    want, bound = table(ids, dY, vocab, scale, pad, old)
    close(dW.check(), want, bound + half_step(DT[wdt]) * want.abs(), "dW")
    if accumulate:   # rows without tokens stay as they were, bit for bit
        met = torch.zeros(vocab, dtype=torch.bool, device=cuda)
        met[ids[ids != pad].long()] = True
        assert torch.equal(dW.t[~met], old[~met])


@pytest.mark.parametrize("tokens", [100, 3000, 20000])
def test_table_gradient_one_id_bad_ids_and_order(cuda, tokens):
    """Every token the same id; ids out of range and padding leave nothing; equal calls, equal bits."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens)
    dY = torch.randn(tokens, 72, generator=g, device=cuda)
    same = torch.full((tokens,), 6, device=cuda)
    dW = torch.empty(7, 72, device=cuda)
    dion.embedding_grad_(same, dY, dW)
    want, bound = table(same, dY, 7, 1.0)
    close(dW, want, bound + 2.0 ** -24 * want.abs(), "one id")
    none = torch.where(torch.arange(tokens, device=cuda) % 2 == 0, -5, 7 + torch.arange(tokens, device=cuda) * (1 << 33))
    dion.embedding_grad_(none, dY, dW)
    assert not dW.any()
    dion.embedding_grad_(same, dY, dW, padding_id=6)
    assert not dW.any()
    dW.fill_(3.0)
    dion.embedding_grad_(same, dY, dW, padding_id=6, accumulate=True)
    assert (dW == 3.0).all()
    ids = skewed_ids(g, tokens, 500, cuda)
    a, b = torch.empty(500, 72, device=cuda), torch.empty(500, 72, device=cuda)
    dion.embedding_grad_(ids, dY, a)
    dion.embedding_grad_(ids, dY, b)
    assert torch.equal(a, b)


def test_table_gradient_matches_differences(cuda):
    """d/dW of sum(dY * lookup(W)): the lookup is linear in W, so a difference of any size is exact up to rounding."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, 5)
    W = torch.randn(30, 16, generator=g, device=cuda)
    ids = torch.randint(0, 30, (200,), generator=g, device=cuda)
    dY = torch.randn(200, 16, generator=g, device=cuda)
    E = torch.randn(30, 16, generator=g, device=cuda)
    dW = dion.embedding_grad_(ids, dY, torch.empty_like(W), 2.0)
    f = lambda X: (dion.embedding_(ids, X, 2.0).double() * dY.double()).sum()   # noqa: E731
    want, got = f(W + E) - f(W - E), 2 * (dW.double() * E.double()).sum()
    assert abs(float(want - got)) <= 1e-5 * float((dY.abs().double().sum(1) * 20).sum()) / 16


# ---------------------------------------------------------------------------- linear cross entropy
HEAD = [(1, 1, 1), (1, 7, 3), (1, 300, 64), (5, 257, 65), (32, 129, 8), (33, 1000, 72), (64, 256, 64), (100, 130, 200),
        (257, 1013, 255), (700, 2048, 128), (1024, 8192, 128), (2048, 300, 4096), (70, 2048, 4160), (3, 40000, 96)]


def head_inputs(g, tokens, vocab, width, dt, device, ignored=0.2):
    W = (torch.randn(vocab, width, generator=g, device=device) * width ** -0.5).to(dt)
    y = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    lean = torch.rand(tokens, 1, generator=g, device=device) * 0.8 * math.log(vocab + 1)
    H = (torch.randn(tokens, width, generator=g, device=device) + lean * W[y].float()).to(dt)
    if tokens > 1:
        y = torch.where(torch.rand(tokens, generator=g, device=device) < ignored, -100, y)
    return H, W, y


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,vocab,width", HEAD)
def test_loss(cuda, tokens, vocab, width, dt):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, vocab, width)
    H, W, y = head_inputs(g, tokens, vocab, width, DT[dt], cuda)
    H[y == -100] = math.nan   # an ignored row may hold anything
    loss, lse = Guarded((tokens,), F32, cuda), Guarded((tokens,), F32, cuda)
    ws = dirty(dion.linear_cross_entropy_workspace_for(tokens, vocab, width, cuda, DT[dt]))
    yy = y.to(torch.int32) if tokens % 2 else y
    dion.linear_cross_entropy_(H, W, yy, loss=loss.t, lse=lse.t, workspace=ws)
    want = Head(H, W, y)
    close(lse.check(), want.lse, want.lse_bound, "lse")
    close(loss.check(), want.loss, want.loss_bound, "loss")


@pytest.mark.parametrize("dt,wdt,accumulate", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "f32", True),
                                               ("f32", "bf16", True)])
@pytest.mark.parametrize("tokens,vocab,width", HEAD)
def test_loss_gradient(cuda, tokens, vocab, width, dt, wdt, accumulate):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, vocab, width, 2)
    H, W, y = head_inputs(g, tokens, vocab, width, DT[dt], cuda)
    H[y == -100] = math.inf
    grad = torch.rand(tokens, generator=g, device=cuda) if tokens % 2 else torch.full((1,), 1.0 / tokens, device=cuda)
    _, lse = dion.linear_cross_entropy_(H, W, y)
    dH, dW = Guarded((tokens, width), DT[dt], cuda), Guarded((vocab, width), DT[wdt], cuda)
    old = None
    if accumulate:
        dW.t.copy_(torch.randn(vocab, width, generator=g, device=cuda) * 0.01)
        old = dW.t.clone()
    ws = dirty(dion.linear_cross_entropy_workspace_for(tokens, vocab, width, cuda, DT[dt], dw_dtype=DT[wdt], for_grad=True))
    dion.linear_cross_entropy_grad_(H, W, y, lse, grad, dH.t, dW.t, accumulate=accumulate, workspace=ws)
    want = Head(H, W, y, grad=grad, dw_dtype=DT[wdt], dw_old=old)
    close(dH.check(), want.dH, want.dH_bound, "dH")
    close(dW.check(), want.dW, want.dW_bound, "dW")
    assert not dH.t[y == -100].any()
    # either gradient alone, and again: the same bits
    dH2, dW2 = torch.empty_like(dH.t), (torch.empty_like(dW.t) if old is None else old.clone())
    dion.linear_cross_entropy_grad_(H, W, y, lse, grad, dH2, None, workspace=None)
    dion.linear_cross_entropy_grad_(H, W, y, lse, grad, None, dW2, accumulate=accumulate)
    if wdt == dt or dt == "f32":
        assert torch.equal(dH2, dH.t)
    assert torch.equal(dW2, dW.t)
