"""GPU tests of the residual blocks' operators together and in their surroundings: a model of them trained through MixedDion
against autograd in 64 bits, captured graphs, several streams, arrays past 32 bits, refusals."""
import pytest
import torch

from tests.block_reference import F64, Ffn, Norm, NormGrad, activation, close, half_step, mask

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def setup_model(device, dt, width=128, hidden=192, vocab=300, layers=2):
    g = torch.Generator(device=device).manual_seed(9)

    def rnd(*s, std=1.0):
        return (torch.randn(*s, generator=g, device=device) * std).to(dt)
    params = [rnd(vocab, width, std=0.05)]   # tied: the embedding and the head
    for _ in range(layers):
        params += [(1 + rnd(width, std=0.1)).to(dt), rnd(hidden, width, std=width ** -0.5), rnd(hidden, width, std=width ** -0.5),
                   rnd(width, hidden, std=hidden ** -0.5)]
    params.append((1 + rnd(width, std=0.1)).to(dt))
    ids = torch.randint(0, vocab, (3, 70), generator=g, device=device)
    targets = torch.randint(0, vocab, (3, 70), generator=g, device=device)
    targets[1, 40:] = -100
    return params, ids, targets


def train(opt, ids, targets, seed, p, layers=2, act="silu", eight=False, keep=True):
    """One forward and backward pass: the stream x, in each layer r = norm(h), y = feed_forward(r), h += dropout(y)."""
    kept, h, y = [], opt.lookup(0, ids, 8.0), None
    for k in range(layers + 1):
        w = 1 + 4 * k
        scale = None
        drop = dict(p=p, seed=seed, site=k) if k else {}
        x, residual = (h, None) if k == 0 else (y, h)
        out = opt.norm(w, x, EPS, eight=eight and k < layers, residual=residual, **drop)
        r, h, rstd = out[0], out[-2], out[-1]
        if eight and k < layers:
            scale = out[1]
        if k < layers:
            y, saved = opt.feed_forward((w + 1, w + 2, w + 3), r, act=act, scale=scale, keep=keep)
            kept.append((r, scale, h, rstd, saved))
        else:
            kept.append((r, None, h, rstd, None))
    loss, dr = opt.head_loss(0, kept[-1][0], targets)
    dh, dy = opt.norm_grad(1 + 4 * layers, dr, kept[-1][2], kept[-1][3], p=p, seed=seed, site=layers)
    for k in reversed(range(layers)):
        r, scale, h, rstd, saved = kept[k]
        w = 1 + 4 * k
        dr = opt.feed_forward_grad((w + 1, w + 2, w + 3), r, dy, saved, act=act, scale=scale)
        drop = dict(p=p, seed=seed, site=k) if k else {}
        dh, dy = opt.norm_grad(w, dr, h, rstd, dsum=dh, **drop)
    opt.lookup_grad(0, ids, dh, 8.0)
    return loss


def reference(params, ids, targets, seed, p, act, layers=2):
    """The same in 64 bits by autograd: (loss per token, gradients)."""
    ws = [q.to(F64).requires_grad_() for q in params]
    h = 8.0 * ws[0][ids]
    y = None
    for k in range(layers + 1):
        w = 1 + 4 * k
        if k:
            keep = mask(h.numel(), p, seed, k, h.device).view(h.shape) if p else torch.ones_like(h)
            h = h + y * keep / (1 - p)
        r = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * ws[w]
        if k < layers:
            v, _, _ = activation(act, r @ ws[w + 1].t())
            y = (v * (r @ ws[w + 2].t())) @ ws[w + 3].t()
    z = (r @ ws[0].t()).reshape(-1, ws[0].shape[0])
    loss = torch.nn.functional.cross_entropy(z, targets.reshape(-1), ignore_index=-100, reduction="none")
    (loss.sum() / (targets != -100).sum()).backward()
    return loss.detach().view(targets.shape), [q.grad for q in ws]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_model_gradients_match_autograd(cuda, p, act):
    """fp32: every gathered gradient is the formula's.  Each of the pass's twenty or so dependent operators keeps its relative
    error (of norms) within a few u sqrt(K), K <= 300 terms, 20 x 2^-24 x 17 x 4 < 1e-4."""
    import rank_orthonormalized_optimizer_amd as dion
    params, ids, targets = setup_model(cuda, F32)
    opt = dion.MixedDion([q.clone() for q in params])
    seed = torch.tensor([77], device=cuda)
    loss = train(opt, ids, targets, seed, p, act=act)
    want, grads = reference(params, ids, targets, 77, p, act)
    assert float((loss.to(F64) - want).abs().max()) < 1e-4 * float(want.abs().max())
    assert opt.pending == set(range(len(params)))
    for i, g in enumerate(grads):
        off = float((opt.gathered[i].to(F64) - g).norm() / g.norm())
        assert off < 1e-4, (i, off)
    # a second microbatch adds, and formed again instead of kept it is the same up to the roundings
    train(opt, ids, targets, seed, p, act=act, keep=False)
    for i, g in enumerate(grads):
        assert float((opt.gathered[i].to(F64) - 2 * g).norm() / g.norm()) < 2e-4, i
    before = [q.clone() for q in opt.params]
    opt.step([None] * len(params))
    assert not opt.pending and all(torch.isfinite(q).all() and not torch.equal(q, b) for q, b in zip(opt.params, before))


@pytest.mark.parametrize("eight", [False, True])
def test_model_in_bf16(cuda, eight):
    """bf16 and with the blocks' input in 8 bits: close to the 64-bit gradients as far as the roundings go, and trains.  A layer
    rounds its stream, its input (8 bits: 2^-4 / sqrt(3) of an element), u and its gradients, about eight roundings of 2^-8 /
    sqrt(3) or, with 8 bits, one of 2^-4 / sqrt(3) that counts, in each of three layers' worth of operators in a row: their norms
    add up to at most 24 x 2^-8 / sqrt(3) = 0.055, and with 8 bits twice 2 x 2^-4 / sqrt(3) = 0.145 besides."""
    import rank_orthonormalized_optimizer_amd as dion
    params, ids, targets = setup_model(cuda, BF16)
    opt = dion.MixedDion([q.clone() for q in params])
    seed = torch.tensor([-5], device=cuda)
    train(opt, ids, targets, seed, 0.1, eight=eight)
    _, grads = reference(params, ids, targets, -5, 0.1, "silu")
    for i, g in enumerate(grads):
        off = float((opt.gathered[i].to(F64) - g).norm() / g.norm())
        assert off < (0.2 if eight else 0.055), (i, off)
    opt.step([None] * len(params))
    assert all(torch.isfinite(q).all() for q in opt.params)


def test_model_pass_in_a_graph(cuda):
    """A captured pass replays with new inputs and a new seed in the same places, each replay as the eager pass, bit for bit."""
    import rank_orthonormalized_optimizer_amd as dion
    for dt in (F32, BF16):
        params, ids, targets = setup_model(cuda, dt)
        seed = torch.tensor([1], device=cuda)
        opt = dion.MixedDion([q.clone() for q in params])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            train(opt, ids, targets, seed, 0.3)
            opt.pending.clear()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss = train(opt, ids, targets, seed, 0.3)
        for i in range(4):
            ids.copy_(ids.roll(7, 1))
            seed.add_(1)
            graph.replay()
            eager = dion.MixedDion([q.clone() for q in params])
            want = train(eager, ids, targets, seed, 0.3)
            torch.cuda.synchronize()
            assert torch.equal(loss, want), (dt, i)
            for k in range(len(params)):
                assert torch.equal(opt.gathered[k], eager.gathered[k]), (dt, i, k)


def calls(cuda, key):
    """Inputs and a pass over every operator."""
    import rank_orthonormalized_optimizer_amd as dion
    g = torch.Generator(device=cuda).manual_seed(key)
    rows, width, hidden = 600 + 40 * key, 320, 1000
    x, r = (torch.randn(rows, width, generator=g, device=cuda).to(BF16) for _ in range(2))
    w = torch.randn(width, generator=g, device=cuda)
    W = [(torch.randn(s, generator=g, device=cuda) / 16).to(BF16) for s in ((hidden, width), (hidden, width), (width, hidden))]
    seed = torch.tensor([key], device=cuda)

    def run(stream=None):
        kw = dict(stream=stream)
        a = dion.dropout_(x, 0.1, seed, 1, residual=r, **kw)
        q, scale, h, rstd = dion.rms_norm_8bit_(a, w, residual=r, p=0.2, seed=seed, **kw)
        gate, up = (torch.empty(rows, hidden, device=cuda, dtype=BF16) for _ in range(2))
        y = dion.gated_ffn_(q, *W, scale=scale, gate=gate, up=up, **kw)
        out = [torch.empty_like(x)] + [torch.empty_like(v) for v in W]
        dion.gated_ffn_grad_(q, *W, y, gate, up, *out, scale=scale, **kw)
        dw = torch.empty_like(w)
        dh, dx = dion.rms_norm_grad_(out[0], h, w, rstd, dw, dsum=y, p=0.2, seed=seed, **kw)
        return [a, q.view(torch.uint8), scale, h, rstd, gate.view(torch.int16), up.view(torch.int16), y, *out, dw, dh, dx]
    return run


def test_calls_on_two_streams_at_once(cuda):
    runs = [calls(cuda, k) for k in (1, 2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        got = []
        for run, stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                got.append(run())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_calls_on_a_given_stream(cuda):
    run = calls(cuda, 3)
    want = run()
    torch.cuda.synchronize()
    got = run(torch.cuda.Stream())   # everything on it, the scratch and the outputs too
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_past_32_bits(cuda):
    """1048576 rows of 4104: element numbers past 2^32 in the arrays and in the mask."""
    import rank_orthonormalized_optimizer_amd as dion
    rows, width, p = 1 << 20, 4104, 0.25
    x = torch.empty(rows, width, device=cuda, dtype=BF16).normal_()
    w = torch.randn(width, device=cuda)
    seed = torch.tensor([12], device=cuda)
    y, h, rstd = dion.rms_norm_(x, w, p=p, seed=seed, site=2)
    some = [slice(a, a + 40) for a in (0, (1 << 31) // width - 20, (1 << 32) // width - 20, rows - 40)]
    for s in some:
        keep = mask(40 * width, p, 12, 2, cuda, s.start * width)
        want = Norm(x[s], w, EPS, None, p, keep)
        close(h[s], want.h, want.h_bound + half_step(BF16) * (want.h.abs() + want.h_bound), "h")
        close(y[s], want.y, want.y_bound + half_step(BF16) * (want.y.abs() + want.y_bound), "y")
    del y
    dh, dx = dion.rms_norm_grad_(x, h, w, rstd, p=p, seed=seed, site=2)
    for s in some:
        keep = mask(40 * width, p, 12, 2, cuda, s.start * width)
        want = NormGrad(x[s], h[s], w, rstd[s], None, p, keep)
        close(dh[s], want.dh, want.dh_bound + half_step(BF16) * (want.dh.abs() + want.dh_bound), "dh")
        close(dx[s], want.dx, want.dx_bound + half_step(BF16) * (want.dx.abs() + want.dx_bound), "dx")
    del dh, dx
    q, scale, _, _ = dion.rms_norm_8bit_(x, w, p=p, seed=seed, site=2, h=h)
    for s in some:
        values, want = Norm(x[s], w, EPS, None, p, mask(40 * width, p, 12, 2, cuda, s.start * width)).eight()
        assert torch.equal(scale[s].to(F64), want) and torch.equal(q[s].to(F64), values)


@pytest.mark.parametrize("t", [F32, BF16])
def test_feed_forward_past_32_bits(cuda, t):
    """20000 rows of 131072 hidden columns: gate, up and u past 2^31 elements (their bytes past 2^32)."""
    import rank_orthonormalized_optimizer_amd as dion
    rows, width, hidden = 20000, 64, 131072
    g = torch.Generator(device=cuda).manual_seed(3)
    X, dY = (torch.randn(rows, width, generator=g, device=cuda).to(t) for _ in range(2))
    Wg, Wu = ((torch.randn(hidden, width, generator=g, device=cuda) / 8).to(t) for _ in range(2))
    Wd = (torch.randn(width, hidden, generator=g, device=cuda) / 362).to(t)
    gate, up = (torch.empty(rows, hidden, device=cuda, dtype=t) for _ in range(2))
    Y = dion.gated_ffn_(X, Wg, Wu, Wd, gate=gate, up=up)
    out = [torch.empty_like(v) for v in (X, Wg, Wu, Wd)]
    dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, gate, up, *out)
    for a in (0, (1 << 31) // hidden - 8, rows - 16):   # some rows, whose outputs are theirs alone
        s = slice(a, a + 16)
        want = Ffn(X[s], Wg, Wu, Wd, "silu")
        close(Y[s], want.Y, want.Y_bound + half_step(t) * (want.Y.abs() + want.Y_bound), "Y")
        want = Ffn(X[s], Wg, Wu, Wd, "silu", None, dY[s], gate[s].contiguous(), up[s].contiguous())
        close(out[0][s], want.dX, want.dX_bound + half_step(t) * (want.dX.abs() + want.dX_bound), "dX")
    for a in (0, hidden - 16):   # some hidden columns, whose weights' gradients are theirs alone
        s = slice(a, a + 16)
        want = Ffn(X, Wg[s], Wu[s], Wd[:, s].contiguous(), "silu", None, dY, gate[:, s].contiguous(), up[:, s].contiguous())
        for k, v in (("dWg", out[1][s]), ("dWu", out[2][s]), ("dWd", out[3][:, s])):
            w, e = getattr(want, k), getattr(want, k + "_bound")
            close(v, w, e + half_step(t) * (w.abs() + e), k)


def test_refusals_on_the_gpu(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    x, w = torch.randn(4, 64, device=cuda), torch.randn(64, device=cuda)
    W, Wd = torch.randn(96, 64, device=cuda), torch.randn(64, 96, device=cuda)
    seed, rstd = torch.tensor([0], device=cuda), torch.ones(4, device=cuda)
    bf = x.to(BF16)
    for call, error in [
            (lambda: dion.dropout_(x, 0.1), ValueError), (lambda: dion.dropout_(x, 1.0, seed), dion.DionError),
            (lambda: dion.dropout_(x, 0.1, seed.int()), TypeError), (lambda: dion.dropout_(x, 0.1, seed.cpu()), ValueError),
            (lambda: dion.dropout_(x, 0.1, torch.zeros(2, dtype=torch.int64, device=cuda)), ValueError),
            (lambda: dion.dropout_(x.t(), 0.1, seed), ValueError), (lambda: dion.dropout_(x, 0.1, seed, residual=x[:3]), ValueError),
            (lambda: dion.dropout_(x, 0.1, seed, residual=x, out=bf), TypeError), (lambda: dion.dropout_(x, 0.1, seed, out=x), dion.DionError),
            (lambda: dion.dropout_(x.double(), 0.1, seed), TypeError), (lambda: dion.rms_norm_(x, w[:63]), ValueError),
            (lambda: dion.rms_norm_(x, w, residual=x.cpu()), ValueError), (lambda: dion.rms_norm_(x, w, residual=bf, h=x), TypeError),
            (lambda: dion.rms_norm_(x, w, -1.0), dion.DionError), (lambda: dion.rms_norm_(x, w, out=x), dion.DionError),
            (lambda: dion.rms_norm_(x, w, out=x.to(torch.float8_e4m3fn)), TypeError), (lambda: dion.rms_norm_8bit_(x, w, out=bf), TypeError),
            (lambda: dion.rms_norm_8bit_(x, w, scale=rstd[:3]), ValueError), (lambda: dion.rms_norm_(torch.ones((), device=cuda), w), ValueError),
            (lambda: dion.rms_norm_grad_(x, x, w, rstd[:3]), ValueError), (lambda: dion.rms_norm_grad_(x, x, w, rstd, dsum=bf), TypeError),
            (lambda: dion.rms_norm_grad_(x, x, w, rstd, p=0.1), ValueError), (lambda: dion.rms_norm_grad_(x, x, w, rstd, dh=bf), TypeError),
            (lambda: dion.rms_norm_grad_(x, x, w, rstd, dx=bf), TypeError), (lambda: dion.rms_norm_grad_(x, x, w, rstd, dh=x), dion.DionError),
            (lambda: dion.gated_ffn_(x, W, W.to(BF16), Wd), TypeError), (lambda: dion.gated_ffn_(x, W, W, Wd.t()), ValueError),
            (lambda: dion.gated_ffn_(x[:, :63].contiguous(), W, W, Wd), ValueError), (lambda: dion.gated_ffn_(bf, W, W, Wd), TypeError),
            (lambda: dion.gated_ffn_(x, W, W, Wd, act="relu"), ValueError), (lambda: dion.gated_ffn_(x, W, W, Wd, scale=rstd), TypeError),
            (lambda: dion.gated_ffn_(x.to(torch.float8_e4m3fn), W, W, Wd), TypeError),
            (lambda: dion.gated_ffn_(x, W, W, Wd, gate=torch.empty(4, 96, device=cuda)), ValueError),
            (lambda: dion.gated_ffn_(x, W, W, Wd, workspace=torch.empty(1, dtype=torch.uint8, device=cuda)), dion.DionError),
            (lambda: dion.gated_ffn_grad_(x, W, W, Wd, x), dion.DionError),
            (lambda: dion.gated_ffn_grad_(x, W, W, Wd, bf, dX=torch.empty_like(x)), TypeError),
            (lambda: dion.gated_ffn_grad_(x, W, W, Wd, x, dWg=torch.empty_like(W)), ValueError),
            (lambda: dion.gated_ffn_grad_(x, W, W, Wd, x, dWg=torch.empty_like(W), dWu=W.to(BF16)), TypeError),
            (lambda: dion.gated_ffn_grad_(x, W, W, Wd, x, dX=x), dion.DionError)]:
        with pytest.raises(error):
            call()
    with pytest.raises(ValueError, match="requires a gradient"):
        dion.rms_norm_(x.clone().requires_grad_(), w)
    misaligned = torch.empty(4 * 64 + 1, device=cuda)[1:].view(4, 64)
    with pytest.raises(dion.DionError):
        dion.rms_norm_(misaligned, w)
    opt = dion.MixedDion([W.clone(), W.clone(), Wd.clone(), w.clone()])
    with pytest.raises(ValueError, match="three"):
        opt.feed_forward((0, 0, 2), x)
    with pytest.raises(ValueError, match="three"):
        opt.feed_forward((0, -4, 2), x)   # the same, counted from the back
    with pytest.raises(IndexError):
        opt.norm(4, x)
    with pytest.raises(ValueError):
        opt.feed_forward_grad((0, 1, 2), x, x[:3])
    assert not opt.pending
    _, kept = opt.feed_forward((0, 1, -2), x)
    opt.feed_forward_grad((0, 1, 2), x, x, kept)
    assert opt.pending == {0, 1, 2}


def test_mixed_dion_adds_where_some_matrices_have_a_gradient(cuda):
    """One of a block's matrices is used twice: the others' gradients start from zero, its own adds up."""
    import rank_orthonormalized_optimizer_amd as dion
    g = torch.Generator(device=cuda).manual_seed(1)
    W = [torch.randn(96, 64, generator=g, device=cuda) / 8 for _ in range(4)] + [torch.randn(64, 96, generator=g, device=cuda) / 8]
    x = torch.randn(50, 64, generator=g, device=cuda)
    opt, a, b = (dion.MixedDion([w.clone() for w in W]) for _ in range(3))
    for o in (opt, a):
        o.feed_forward_grad((0, 1, 4), x, x)
    for o in (opt, b):
        o.feed_forward_grad((2, 1, 4), x, x)
    for i in (0, 1, 2, 4):
        want = sum(o.gathered[i].to(F64) for o in (a, b) if i in o.pending)
        assert float((opt.gathered[i].to(F64) - want).abs().max()) <= 4 * 2.0 ** -24 * float(want.abs().max()), i
