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
                                                (70, 31, 4104), (1030, 50, 255), (130, 33, 1301), (129, 40, 1023)])
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
        (257, 1013, 255), (700, 2048, 128), (1024, 8192, 128), (2048, 300, 4096), (70, 2048, 4160), (3, 40000, 96),
        (1, 16384, 3), (5, 20011, 70), (33, 16500, 133), (128, 16385, 65)]   # fp32: W read in place, rows of any length
HEAD += [(1, 1030, 700), (20, 2000, 1290), (129, 1500, 1000), (300, 257, 2100), (33, 12347, 1100), (1198, 1640, 770)]   # sliced logits


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


# sizes that go through several pieces of the vocabulary: D's bytes (many tokens), W's planes (wide fp32), D of few tokens
@pytest.mark.parametrize("tokens,vocab,width,dt", [(32768, 9000, 24, "f32"), (65536, 5000, 32, "bf16"), (100001, 300, 16, "bf16"),
                                                   (65536, 9000, 32, "bf16"), (200001, 8000, 16, "bf16"),
                                                   (200, 140000, 4096, "f32"),
                                                   (3, 1100000, 8, "f32"), (193, 9000, 68, "f32"), (192, 9000, 68, "f32")])
def test_pieces_of_the_vocabulary(cuda, tokens, vocab, width, dt):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, vocab, width, 3)
    H, W, y = head_inputs(g, tokens, vocab, width, DT[dt], cuda)
    grad = torch.rand(tokens, generator=g, device=cuda)
    loss, lse = dion.linear_cross_entropy_(H, W, y)
    dH, dW = Guarded(H.shape, DT[dt], cuda), Guarded(W.shape, DT[dt], cuda)
    ws = dirty(dion.linear_cross_entropy_workspace_for(tokens, vocab, width, cuda, DT[dt], for_grad=True))
    dion.linear_cross_entropy_grad_(H, W, y, lse, grad, dH.t, dW.t, workspace=ws)
    want = Head(H, W, y, grad=grad)
    close(loss, want.loss, want.loss_bound, "loss")
    close(dH.check(), want.dH, want.dH_bound, "dH")
    close(dW.check(), want.dW, want.dW_bound, "dW")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [20, 300])
def test_ignored_and_bad_targets(cuda, tokens, dt):
    """All ignored: nothing; another ignore_index; targets out of range make NaN of their own loss and row, and of dW."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, 4)
    H, W, y = head_inputs(g, tokens, 50, 40, DT[dt], cuda, ignored=0)
    one = torch.ones(1, device=cuda)
    none = torch.full_like(y, -100)
    loss, lse = dion.linear_cross_entropy_(H, W, none)
    assert not loss.any() and not lse.any()
    dH, dW = torch.full_like(H, 3), torch.full_like(W, 3)
    dion.linear_cross_entropy_grad_(H, W, none, lse, one, dH, dW, accumulate=True)
    assert not dH.any() and (dW == 3).all()
    dion.linear_cross_entropy_grad_(H, W, none, lse, one, dH, dW)
    assert not dW.any()
    # the targets of id 0 ignored, as padding
    y[::3] = 0
    loss, lse = dion.linear_cross_entropy_(H, W, y, ignore_index=0)
    dion.linear_cross_entropy_grad_(H, W, y, lse, one, dH, dW, ignore_index=0)
    want = Head(H, W, y, ignore=0, grad=one)
    close(loss, want.loss, want.loss_bound, "loss")
    close(dH, want.dH, want.dH_bound, "dH")
    close(dW, want.dW, want.dW_bound, "dW")
    y[1], y[2] = 50, -7
    y[4] = 1 << 40
    loss, lse = dion.linear_cross_entropy_(H, W, y, ignore_index=0)
    dion.linear_cross_entropy_grad_(H, W, y, lse, one, dH, dW, ignore_index=0)
    want = Head(H, W, y, ignore=0, grad=one)
    close(loss, want.loss, want.loss_bound, "loss")
    close(lse, want.lse, want.lse_bound, "lse")
    close(dH, want.dH, want.dH_bound, "dH")
    assert torch.isnan(dW).all()


@pytest.mark.parametrize("tokens", [30, 400])
def test_fp32_rows_of_any_scale(cuda, tokens):
    """Rows from 2^-60 up, zero rows among them: fp32 logits stay accurate relative to each row's own terms."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, 5)
    H, W, y = head_inputs(g, tokens, 700, 136, F32, cuda)
    H *= torch.exp2(torch.randint(-60, 1, (tokens, 1), generator=g, device=cuda).float())
    W *= torch.exp2(torch.randint(-40, 1, (700, 1), generator=g, device=cuda).float())
    H[3], W[5] = 0, 0
    grad = torch.ones(1, device=cuda)
    loss, lse = dion.linear_cross_entropy_(H, W, y)
    dH, dW = torch.empty_like(H), torch.empty_like(W)
    dion.linear_cross_entropy_grad_(H, W, y, lse, grad, dH, dW)
    want = Head(H, W, y, grad=grad)
    close(loss, want.loss, want.loss_bound, "loss")
    close(dH, want.dH, want.dH_bound, "dH")
    close(dW, want.dW, want.dW_bound, "dW")


@pytest.mark.parametrize("vocab,scale", [(300, 2.0 ** -30), (300, 1.0), (1000, 2.0 ** 20)])
def test_fp32_padded_vocabulary(cuda, vocab, scale):
    """Rows of zeros behind the true vocabulary take nothing from the others' precision, whatever their size."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, vocab, 11)
    H, W, y = head_inputs(g, 200, vocab, 72, F32, cuda)
    H /= scale
    W *= scale
    W[vocab - 60:] = 0
    grad = torch.rand(200, generator=g, device=cuda) * 2.0 ** -20
    loss, lse = dion.linear_cross_entropy_(H, W, y)
    dH, dW = torch.empty_like(H), torch.empty_like(W)
    dion.linear_cross_entropy_grad_(H, W, y, lse, grad, dH, dW)
    want = Head(H, W, y, grad=grad)
    close(loss, want.loss, want.loss_bound, "loss")
    close(dH, want.dH, want.dH_bound, "dH")
    close(dW, want.dW, want.dW_bound, "dW")


@pytest.mark.parametrize("tokens", [24, 260])
def test_loss_gradient_matches_differences(cuda, tokens):
    """Central differences of the summed loss along a direction in H and W.  With a = the largest change of a logit per
    unit step, the third derivative of a token's loss is at most (2 a)^3: the difference is off by eps^2 (2 a)^3 / 6,
    plus the two losses' own errors over 2 eps."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, tokens, 6)
    H, W, y = head_inputs(g, tokens, 300, 64, F32, cuda)
    for which in ("H", "W"):
        E = torch.randn((H if which == "H" else W).shape, generator=g, device=cuda) * 0.05
        eps = 0.0625
        X = H if which == "H" else W

        def f(sign):
            Z = X + sign * eps * E
            a, b = (Z, W) if which == "H" else (H, Z)
            want = Head(a, b, y)
            return dion.linear_cross_entropy_(a, b, y)[0].double().sum(), want.loss_bound.sum()

        (up, e1), (down, e2) = f(1), f(-1)
        loss, lse = dion.linear_cross_entropy_(H, W, y)
        dH, dW = torch.empty_like(H), torch.empty_like(W)
        dion.linear_cross_entropy_grad_(H, W, y, lse, torch.ones(1, device=cuda), dH, dW)
        got = ((dH if which == "H" else dW).double() * E.double()).sum()
        rate = (E.double() @ W.double().t() if which == "H" else H.double() @ E.double().t()).abs().amax(1)
        bound = (eps ** 2 * (2 * rate) ** 3 / 6).sum() + (e1 + e2) / (2 * eps)
        exact = Head(H, W, y, grad=torch.ones(1, device=cuda))
        bound = bound + ((exact.dH_bound if which == "H" else exact.dW_bound) * E.double().abs()).sum()
        # X + eps E is rounded to fp32 once: half a step of X times the gradient, over 2 eps
        slope = (exact.dH if which == "H" else exact.dW).abs()
        bound = bound + 2 * (2.0 ** -24 * (X.double().abs() + eps * E.double().abs()) * slope).sum() / (2 * eps)
        assert abs(float((up - down) / (2 * eps) - got)) <= float(bound)


def test_offsets_past_32_bits(cuda):
    """A table of 2.46e9 elements: its last rows looked up, its gradient written, its logits formed."""
    import rank_orthonormalized_optimizer_amd as dion
    vocab, width = 600001, 4096
    g = gen(cuda, 7)
    W = torch.empty(vocab, width, dtype=BF16, device=cuda)
    for a in range(0, vocab, 100000):
        W[a:a + 100000] = torch.randn(W[a:a + 100000].shape, generator=g, device=cuda) / 64
    ids = torch.tensor([vocab - 1, 0, vocab - 2, 524288, vocab - 1, 524287], device=cuda)
    assert torch.equal(dion.embedding_(ids, W, 2.0), W[ids] * 2)
    dY = torch.randn(6, width, generator=g, device=cuda).to(BF16)
    dW = torch.full_like(W, 5)
    dion.embedding_grad_(ids, dY, dW)
    rows = torch.zeros(vocab, dtype=torch.bool, device=cuda)
    rows[ids] = True
    assert not dW[~rows].any()
    want = dY.double()
    want[0] += want[4]
    for k in (0, 1, 2, 3, 5):
        assert torch.equal(dW[ids[k]], want[k].to(BF16))
    H = torch.randn(6, width, generator=g, device=cuda).to(BF16)
    loss, lse = dion.linear_cross_entropy_(H, W, ids)
    z = torch.cat([H.double() @ W[a:a + 50000].double().t() for a in range(0, vocab, 50000)], 1)
    true = torch.logsumexp(z, 1)
    size = torch.cat([H.double().abs() @ W[a:a + 50000].double().abs().t() for a in range(0, vocab, 50000)], 1).amax(1)
    bound = 2 * (2 * width + 12) * 2.0 ** -24 * size + (96 + vocab / 64 + 8) * 2.0 ** -24 + 4 * 2.0 ** -24 * true
    close(lse, true, bound, "lse")
    close(loss, true - z[torch.arange(6, device=cuda), ids], bound, "loss")
    dH = torch.empty_like(H)
    dion.linear_cross_entropy_grad_(H, W, ids, lse, torch.ones(1, device=cuda), dH, dW)
    D = torch.exp(z - true[:, None])
    D[torch.arange(6, device=cuda), ids] -= 1
    for a in (0, 524280, vocab - 8):
        part = D[:, a:a + 8].t() @ H.double()
        e = (2 * (2 * width + 12) * 2.0 ** -24 * size.max() + vocab / 64 * 2.0 ** -24 + 2.0 ** -8 + 2.0 ** -16)
        close(dW[a:a + 8], part, e * (torch.exp(z - true[:, None])[:, a:a + 8].t() + D[:, a:a + 8].abs().t()) @ H.double().abs()
              + 2.0 ** -8 * part.abs(), "dW")


# ---------------------------------------------------------------------------- together
def _everything(dion, s, out):
    """Lookup, loss, its gradients, table gradient on top of the head's: one tied step."""
    h = dion.embedding_(s["ids"], s["W"], 4.0, out["h"])
    dion.linear_cross_entropy_(h, s["W"], s["y"], loss=out["loss"], lse=out["lse"], workspace=out["w1"])
    dion.linear_cross_entropy_grad_(h, s["W"], s["y"], out["lse"], s["g"], out["dH"], out["dW"], workspace=out["w2"])
    dion.embedding_grad_(s["ids"], out["dH"], out["dW"], 4.0, padding_id=0, accumulate=True, workspace=out["w3"])


def _state(dion, cuda, key, tokens, vocab, width, dt):
    g = gen(cuda, 8, key)
    s = {"W": (torch.randn(vocab, width, generator=g, device=cuda) / 8).to(dt), "ids": skewed_ids(g, tokens, vocab, cuda),
         "y": skewed_ids(g, tokens, vocab, cuda), "g": torch.full((1,), 1.0 / tokens, device=cuda)}
    s["y"][::5] = -100
    return s


def _outputs(dion, cuda, tokens, vocab, width, dt):
    e = lambda *shape, t=dt: torch.empty(shape, dtype=t, device=cuda)   # noqa: E731
    return {"h": e(tokens, width), "loss": e(tokens, t=F32), "lse": e(tokens, t=F32), "dH": e(tokens, width), "dW": e(vocab, width),
            "w1": dion.linear_cross_entropy_workspace_for(tokens, vocab, width, cuda, dt),
            "w2": dion.linear_cross_entropy_workspace_for(tokens, vocab, width, cuda, dt, for_grad=True),
            "w3": dion.embedding_grad_workspace_for(tokens, vocab, width, cuda)}


RESULTS = ("h", "loss", "lse", "dH", "dW")


@pytest.mark.parametrize("tokens,vocab,width,dt", [(40, 300, 64, BF16), (700, 1000, 128, F32), (20000, 500, 72, BF16)])
def test_graph_replays_match_eager_calls(cuda, tokens, vocab, width, dt):
    """One captured step, replayed on new inputs with eager work and synchronizations between the replays."""
    import rank_orthonormalized_optimizer_amd as dion
    states = [_state(dion, cuda, k, tokens, vocab, width, dt) for k in range(3)]
    want = []
    for s in states:
        out = _outputs(dion, cuda, tokens, vocab, width, dt)
        _everything(dion, s, out)
        torch.cuda.synchronize()
        want.append({k: out[k].clone() for k in RESULTS})
    held = {k: v.clone() for k, v in states[0].items()}
    out = _outputs(dion, cuda, tokens, vocab, width, dt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(dion, held, out)
    for k in (1, 0, 2, 1):
        for name in held:
            held[name].copy_(states[k][name])
        for name in ("w1", "w2", "w3"):
            dirty(out[name])
        graph.replay()
        eager = _outputs(dion, cuda, tokens, vocab, width, dt)
        _everything(dion, states[(k + 1) % 3], eager)
        torch.cuda.synchronize()
        for name in RESULTS:
            assert torch.equal(out[name], want[k][name]), f"replay {k}: {name}"
            assert torch.equal(eager[name], want[(k + 1) % 3][name]), f"beside replay {k}: {name}"


def test_calls_on_two_streams_at_once(cuda):
    """Calls on side streams with scratch allocated inside them, beside each other and beside work on the current stream."""
    import rank_orthonormalized_optimizer_amd as dion
    tokens, vocab, width = 600, 4000, 256
    states = [_state(dion, cuda, k, tokens, vocab, width, BF16) for k in range(2)]

    def run(s, stream=None):
        loss, lse = dion.linear_cross_entropy_(s["H"], s["W"], s["y"], stream=stream)
        dH, dW = torch.empty_like(s["H"]), torch.empty_like(s["W"])
        dion.linear_cross_entropy_grad_(s["H"], s["W"], s["y"], lse, s["g"], dH, dW, stream=stream)
        dion.embedding_grad_(s["ids"], dH, dW, accumulate=True, stream=stream)
        return loss, lse, dH, dW, dion.embedding_(s["ids"], dW, stream=stream)

    for s in states:
        s["H"] = dion.embedding_(s["ids"], s["W"])
    want = [run(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(4):
        got = [run(s, st) for s, st in zip(states, streams)]
        here = run(states[0])
        torch.cuda.synchronize()
        for a, b in zip(got + [here], want + [want[0]]):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals_on_the_gpu(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    W, H = torch.zeros(10, 16, device=cuda), torch.zeros(4, 16, device=cuda)
    ids = torch.zeros(4, dtype=torch.int64, device=cuda)
    one = torch.ones(1, device=cuda)
    with pytest.raises(ValueError, match="contiguous"):
        dion.embedding_(ids, W[:, ::2])
    with pytest.raises(TypeError, match="dtype"):
        dion.embedding_(ids.float(), W)
    with pytest.raises(TypeError, match="dtype"):
        dion.embedding_(ids, W.double())
    with pytest.raises(ValueError, match="shape"):
        dion.embedding_(ids, W, out=torch.empty(4, 17, device=cuda))
    with pytest.raises(ValueError, match="matrix"):
        dion.embedding_(ids, W[0])
    with pytest.raises(dion.DionError) as e:
        dion.embedding_(ids, W.view(-1)[4:148].view(9, 16))     # 16 bytes in: accepted alignment
        dion.embedding_(ids, W.view(-1)[1:145].view(9, 16))
    assert e.value.status == -5
    with pytest.raises(ValueError, match="shape"):
        dion.embedding_grad_(ids, H[:3], W)
    with pytest.raises(TypeError, match="dtype"):
        dion.linear_cross_entropy_(H.to(BF16), W, ids)
    with pytest.raises(ValueError, match="shape"):
        dion.linear_cross_entropy_(H, W, ids[:3])
    with pytest.raises(ValueError, match="CPU|cpu|GPU"):
        dion.linear_cross_entropy_(H, W, ids.cpu())
    loss, lse = dion.linear_cross_entropy_(H, W, ids)
    with pytest.raises(ValueError, match="one element"):
        dion.linear_cross_entropy_grad_(H, W, ids, lse, torch.ones(2, device=cuda), torch.empty_like(H))
    with pytest.raises(dion.DionError) as e:
        dion.linear_cross_entropy_grad_(H, W, ids, lse, one)
    assert e.value.status == -1
    with pytest.raises(dion.DionError) as e:
        dion.linear_cross_entropy_grad_(H, W, ids, lse, one, H)
    assert e.value.status == -6
    with pytest.raises(dion.DionError) as e:
        dion.embedding_grad_(ids, H, W, workspace=torch.empty(256, dtype=torch.uint8, device=cuda))
    assert e.value.status == -7


def test_empty_batches(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    W, ids = torch.ones(9, 24, device=cuda), torch.zeros(0, 3, dtype=torch.int32, device=cuda)
    H = dion.embedding_(ids, W)
    assert H.shape == (0, 3, 24)
    loss, lse = dion.linear_cross_entropy_(H, W, ids)
    assert loss.shape == lse.shape == (0, 3)
    dW = torch.ones_like(W)
    dion.linear_cross_entropy_grad_(H, W, ids, lse, torch.ones(1, device=cuda), torch.empty_like(H), dW, accumulate=True)
    dion.embedding_grad_(ids, H, dW, accumulate=True)
    assert (dW == 1).all()
    dion.linear_cross_entropy_grad_(H, W, ids, lse, torch.ones(1, device=cuda), None, dW)
    assert not dW.any()
    dW.fill_(1)
    dion.embedding_grad_(ids, H, dW)
    assert not dW.any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("other", ["adamw", "lion"])
def test_mixed_dion_trains_a_tied_model(cuda, dt, other):
    """One tied matrix and one hidden layer through MixedDion, two microbatches a step: the gathered gradient is the one of
    the formula, and step() with it equals step() with the same gradient given."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, 9)
    vocab, width, scale = 300, 64, 8.0
    table_ = (torch.randn(vocab, width, generator=g, device=cuda) / 8).to(dt)
    layer = (torch.randn(width, width, generator=g, device=cuda) / 8).to(dt)
    bias = torch.zeros(width, dtype=dt, device=cuda)
    a = dion.MixedDion([table_.clone(), layer.clone(), bias.clone()], other=other)
    b = dion.MixedDion([table_.clone(), layer.clone(), bias.clone()], other=other)
    batches = [(skewed_ids(g, 48, vocab, cuda).view(4, 12), skewed_ids(g, 48, vocab, cuda).view(4, 12)) for _ in range(4)]
    for step in range(2):
        W, L, c = (p.detach().double() for p in a.params)
        dL, dc = torch.zeros_like(a.params[1]), torch.zeros_like(a.params[2])
        Wd = W.clone().requires_grad_()
        for ids, y in batches[2 * step:2 * step + 2]:
            y = torch.where(y % 7 == 0, -100, y)
            h = a.lookup(0, ids, scale)
            H = torch.addmm(a.params[2], h.view(-1, width), a.params[1]).view(h.shape)
            loss, dH = a.head_loss(0, H, y)
            dh = (dH.view(-1, width) @ a.params[1].t().contiguous()).view(h.shape)
            dL += h.view(-1, width).t().contiguous() @ dH.view(-1, width)
            dc += dH.sum((0, 1))
            a.lookup_grad(0, ids, dh, scale)
            z = ((Wd[ids] * scale) @ L + c) @ Wd.t()
            ref = torch.nn.functional.cross_entropy(z.view(-1, vocab), y.reshape(-1), ignore_index=-100)
            ref.backward()
            ref = ref.detach()
            # the hidden states are rounded to dt between the operators: a few roundings of the loss's size
            counted = loss[y != -100].double().mean()
            assert abs(float(counted - ref)) <= 16 * torch.finfo(dt).eps * float(ref)
        got = a.gathered[0].double()
        # each of the at most 64 roundings between table and loss gives a relative 2^-24 or 2^-8 of the gradient's own scale
        assert float((got - Wd.grad).norm()) <= 64 * torch.finfo(dt).eps / 2 * float(Wd.grad.norm())
        given = [a.gathered[0].clone(), dL, dc]
        a.step([None, dL, dc])
        b.step(given)
        torch.cuda.synchronize()
        for p, q in zip(a.params, b.params):
            assert torch.equal(p, q)
    with pytest.raises(ValueError, match="no gradient"):
        a.step([None, dL, dc])
    a.head_loss(0, H, y)
    with pytest.raises(ValueError, match="gathered"):
        a.step(given)
