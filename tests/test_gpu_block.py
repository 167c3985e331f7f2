"""GPU tests of the residual blocks' operators (dropout, RMS norm with the residual's addition and in 8
bits, the gated feed-forward block, and their gradients) against their definitions in 64 bits, at the
sizes where they can go wrong.  Every output lies between canaries that must survive, and every
workspace starts out filled with NaN bit patterns."""
import pytest
import torch

from tests.block_reference import (F64, Ffn, Guarded, Norm, NormGrad, close, dirty, half_step, keep, keep_step, kept,
                                   mask)

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DT = {"f32": F32, "bf16": BF16}
EPS = 1e-6


def gen(device, *key):
    seed = 23
    for k in key:
        seed = seed * 1000003 + int(k)
    return torch.Generator(device=device).manual_seed(seed % (1 << 62))


def rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(dtype)


def a_seed(value, device):
    return torch.tensor([value], dtype=torch.int64, device=device)


SEEDS = [0, 1, -1, 0x123456789abcdef, -(1 << 63)]


# ---------------------------------------------------------------------------- dropout
@pytest.mark.parametrize("xdt,odt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [0, 1, 3, 4, 5, 8, 9, 255, 2048, 65537, 1 << 20])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_dropout(cuda, n, p, xdt, odt):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, n, int(p * 1000))
    seed, site = SEEDS[n % len(SEEDS)], [0, 7, -3, 1 << 40][n % 4]
    x, r = rand(g, (n,), DT[xdt]), rand(g, (n,), DT[odt])
    keep = mask(n, p, seed, site, cuda)
    for residual in (None, r):
        out = Guarded((n,), DT[odt], cuda)
        assert dion.dropout_(x, p, a_seed(seed, cuda), site, residual=residual, out=out.t) is out.t
        want = torch.where(keep, x.to(F64), 0.0) / (1 - p)
        bound = 2 * 2.0 ** -24 * want.abs()
        if residual is not None:
            want = want + r.to(F64)
            bound = bound + 2.0 ** -24 * want.abs()
        close(out.check(), want, 1.01 * (bound + half_step(DT[odt]) * want.abs()), "dropout")
    into = Guarded((n,), DT[odt], cuda)   # in place
    into.t.copy_(r)
    dion.dropout_(x, p, a_seed(seed, cuda), site, residual=into.t, out=into.t)
    assert torch.equal(into.check(), out.t)
    if n >= 65537 and 0 < p:
        kept = float(keep.double().mean())
        assert abs(kept - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5


def test_dropout_known_answers(cuda):
    """Philox4x32-10's published words for a counter and key of zeros."""
    import rank_orthonormalized_optimizer_amd as dion
    words = torch.tensor([0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8], dtype=F64, device=cuda)
    for e in range(4):   # the word is where keeping begins
        for step, kept in ((0.0, True), (1.0, False)):
            out = dion.dropout_(torch.ones(4, device=cuda), float((words[e] + step) / 2 ** 32), a_seed(0, cuda))
            assert bool(out[e] != 0) is kept


def test_dropout_past_32_bits(cuda):
    """Elements behind number 2^32 of an array of more."""
    import rank_orthonormalized_optimizer_amd as dion
    x = torch.ones((1 << 32) + 4099, dtype=BF16, device=cuda)
    out = dion.dropout_(x, 0.5, a_seed(5, cuda), 1)
    for start in (0, 1 << 31, 1 << 32):
        assert torch.equal(out[start:start + 4099] != 0, mask(4099, 0.5, 5, 1, cuda, start))


# ---------------------------------------------------------------------------- norm
ROWS = [(1, 1), (3, 7), (5, 8), (2, 64), (70, 255), (9, 512), (6, 513), (5, 1001), (33, 1024), (4, 1032), (3, 2048), (7, 2050),
        (2, 4096), (3, 5001), (2, 8192), (3, 8200), (2, 16384), (2, 20001), (1, 40000), (2, 65536), (1300, 136)]


@pytest.mark.parametrize("xdt,sdt,wdt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                         ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("rows,width", ROWS)
def test_norm(cuda, rows, width, xdt, sdt, wdt):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, rows, width)
    x, r, w = rand(g, (rows, width), DT[xdt]), rand(g, (rows, width), DT[sdt], 3.0), rand(g, (width,), DT[wdt])
    seed, site = a_seed(-77, cuda), 3
    for p in (0.0, 0.2):
        keep = mask(rows * width, p, -77, site, cuda) if p else None
        want = Norm(x, w, EPS, r, p, keep)
        h, y = Guarded((rows, width), DT[sdt], cuda), Guarded((rows, width), DT[xdt], cuda)
        rstd = Guarded((rows,), F32, cuda)
        got = dion.rms_norm_(x, w, EPS, residual=r, p=p, seed=seed, site=site, h=h.t, out=y.t, rstd=rstd.t)
        assert got[0] is y.t and got[1] is h.t and got[2] is rstd.t
        close(h.check(), want.h, want.h_bound + half_step(DT[sdt]) * (want.h.abs() + want.h_bound), "h")
        close(rstd.check(), want.rstd, want.rstd_bound, "rstd")
        close(y.check(), want.y, want.y_bound + half_step(DT[xdt]) * (want.y.abs() + want.y_bound), "y")
        values, scale = want.eight()
        q, s, rstd8 = Guarded((rows, width), E4M3, cuda), Guarded((rows,), F32, cuda), Guarded((rows,), F32, cuda)
        h8 = Guarded((rows, width), DT[sdt], cuda)
        got = dion.rms_norm_8bit_(x, w, EPS, residual=r, p=p, seed=seed, site=site, h=h8.t, out=q.t, scale=s.t, rstd=rstd8.t)
        assert got[0] is q.t and got[1] is s.t and got[2] is h8.t and got[3] is rstd8.t
        assert torch.equal(s.check().to(F64), scale)
        assert torch.equal(q.check().to(F64), values)
        close(rstd8.check(), want.rstd, half_step(F32) * 1.01 * want.rstd, "rstd of 8 bits")
        assert torch.equal(h8.check().to(F64), want.h.to(DT[sdt]).to(F64) if sdt == "f32" else h8.t.to(F64))
        close(h8.t, want.h, half_step(DT[sdt]) * 1.0001 * want.h.abs(), "h of 8 bits")
        into = Guarded((rows, width), DT[sdt], cuda)   # the stream in place
        into.t.copy_(r)
        dion.rms_norm_(x, w, EPS, residual=into.t, p=p, seed=seed, site=site, h=into.t)
        assert torch.equal(into.check(), h.t)


def test_norm_alone_and_its_other_types(cuda):
    """Neither residual nor dropout: h is x; y in another type than x; widths with one element."""
    import rank_orthonormalized_optimizer_amd as dion
    x, w = torch.randn(2, 3, 40, device=cuda, dtype=BF16), torch.randn(40, device=cuda)
    y = torch.empty(2, 3, 40, device=cuda)
    got, h, rstd = dion.rms_norm_(x, w, EPS, out=y)
    assert h is x and got is y and rstd.shape == (2, 3)
    want = Norm(x, w, EPS)
    close(y, want.y, want.y_bound + half_step(F32) * want.y.abs(), "y")
    y, h, rstd = dion.rms_norm_(x, w, EPS, h=torch.empty(2, 3, 40, device=cuda))
    assert torch.equal(h, x.float()) and y.dtype == BF16
    for empty in (dion.rms_norm_(x[:0], w), dion.rms_norm_8bit_(x[:0], w)):
        assert all(t.numel() == 0 for t in empty)


def test_norm_zeros_infinities_and_tiny_rows(cuda):
    """Rows of zeros, of the smallest and the largest numbers, with an infinity or a NaN: the others' rows stay as they are."""
    import rank_orthonormalized_optimizer_amd as dion
    x = torch.randn(7, 96, device=cuda)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, 5] = float("inf")
    x[5, 6] = float("nan")
    x[6, 0] = 448 * 2.0 ** -9
    w = torch.ones(96, device=cuda)
    y, _, rstd = dion.rms_norm_(x, w, EPS)
    want = Norm(x, w, EPS)
    for i in (0, 1, 2, 3, 6):
        close(y[i:i + 1], want.y[i:i + 1], want.y_bound[i:i + 1] + half_step(F32) * want.y[i:i + 1].abs() + 2.0 ** -126, "y")
    assert torch.isnan(y[4, 5]) and (y[4, :5] == 0).all() and torch.isnan(y[5]).all()
    q, scale, _, _ = dion.rms_norm_8bit_(x, w, EPS)
    values, s = want.eight()
    for i in (0, 1, 2, 3, 6):
        assert torch.equal(q[i].to(F64), values[i]) and float(scale[i]) == float(s[i])
    assert torch.isnan(q[4, 5].float()) and (q[4, :5].float() == 0).all() and float(scale[4]) == 1
    assert torch.isnan(q[5].float()).all() and float(scale[5]) == 1


def test_eight_bits_at_their_borders(cuda):
    """Values on and next to the borders between 8-bit numbers, and a largest value on and next to the scale's border."""
    import rank_orthonormalized_optimizer_amd as dion
    width = 512
    grid = torch.arange(0, 127, device=cuda, dtype=torch.uint8).view(E4M3).to(F64)   # 0 .. 448
    ties = (grid[1:] + grid[:-1]) / 2
    row = torch.cat([grid[1:], ties, -ties, torch.nextafter(ties.float(), torch.zeros(1, device=cuda)).to(F64)])[:width]
    row = torch.cat([row, torch.zeros(width - row.numel(), dtype=F64, device=cuda)])
    for top in (448.0, 447.9999, 448.00003, 224.0, 224.00002, 1.75, 1.7500001):
        x = (row / 448 * top).float()[None]
        want = Norm(x, torch.ones(width, device=cuda), 0.0)
        # a weight that undoes the norm up to fp32: values stay next to their borders
        w = torch.full((width,), float(1 / want.rstd[0]), device=cuda)
        want = Norm(x, w, 0.0)
        q, scale, _, _ = dion.rms_norm_8bit_(x, w, 0.0)
        values, s = want.eight()
        assert torch.equal(scale.to(F64), s)
        near = (want.y / s[:, None] - values).abs() / torch.exp2((torch.frexp(values.abs().clamp(min=2 ** -6))[1] - 5).to(F64))
        off = q.to(F64) != values
        assert not bool((off & (near < 1 - 1e-9)).any())   # equal but where 64 bits cannot tell


# ---------------------------------------------------------------------------- norm's gradients
@pytest.mark.parametrize("ydt,sdt,wdt,accumulate", [("f32", "f32", "f32", False), ("bf16", "bf16", "bf16", False),
                                                    ("bf16", "f32", "f32", True), ("f32", "bf16", "bf16", True)])
@pytest.mark.parametrize("rows,width", ROWS + [(0, 40), (5000, 24), (1030, 2056)])
def test_norm_gradients(cuda, rows, width, ydt, sdt, wdt, accumulate):
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, rows, width, 2)
    h, dY, w = rand(g, (rows, width), DT[sdt], 3.0), rand(g, (rows, width), DT[ydt]), rand(g, (width,), DT[wdt])
    s = rand(g, (rows, width), DT[sdt])
    rstd = Norm(h, w, EPS).rstd.float()
    seed, site = a_seed(99, cuda), -5
    for p, dsum in ((0.0, None), (0.3, s)):
        keep = mask(rows * width, p, 99, site, cuda) if p else None
        dw = Guarded((width,), DT[wdt], cuda)
        if accumulate:
            dw.t.copy_(rand(g, (width,), F32))
        want = NormGrad(dY, h, w, rstd, dsum, p, keep, dw.t.clone() if accumulate else None)
        dh, dx = Guarded((rows, width), DT[sdt], cuda), Guarded((rows, width), DT[ydt], cuda)
        ws = dirty(dion.rms_norm_grad_workspace_for(rows, width, cuda))
        got = dion.rms_norm_grad_(dY, h, w, rstd, dw.t, dsum=dsum, p=p, seed=seed, site=site, dh=dh.t, dx=dx.t,
                                  accumulate=accumulate, workspace=ws)
        assert got[0] is dh.t and got[1] is dx.t
        close(dh.check(), want.dh, want.dh_bound + half_step(DT[sdt]) * (want.dh.abs() + want.dh_bound), "dh")
        close(dx.check(), want.dx, want.dx_bound + half_step(DT[ydt]) * (want.dx.abs() + want.dx_bound), "dx")
        close(dw.check(), want.dw, want.dw_bound + half_step(DT[wdt]) * (want.dw.abs() + want.dw_bound), "dw")
        if dsum is not None:   # in place, and without dw and dx
            into = Guarded((rows, width), DT[sdt], cuda)
            into.t.copy_(s)
            dion.rms_norm_grad_(dY, h, w, rstd, dsum=into.t, dh=into.t)
            assert torch.equal(into.check(), dh.t)
    a, b = dion.rms_norm_grad_(dY, h, w, rstd)
    assert a is b


def test_norm_gradient_by_differences(cuda):
    """dh, dx and dw of sum(c y) + sum(e h) against differences of the 64-bit definition."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, 5)
    rows, width, p, site = 4, 12, 0.25, 9
    x, r, w = (rand(g, s, F32).to(F64) for s in ((rows, width), (rows, width), (width,)))
    c, e = rand(g, (rows, width), F32).to(F64), rand(g, (rows, width), F32).to(F64)
    keep = mask(rows * width, p, 11, site, cuda)

    def value(x, r, w):
        n = Norm(x, w, EPS, r, p, keep)
        return float((c * n.y + e * n.h).sum())
    n = Norm(x, w, EPS, r, p, keep)
    dw = torch.empty(width, device=cuda)
    dh, dx = dion.rms_norm_grad_(c.float(), n.h.float(), w.float(), n.rstd.float(), dw, dsum=e.float(), p=p, seed=a_seed(11, cuda),
                                 site=site)
    step = 1e-5
    for what, arg, grad in (("x", 0, dx), ("residual", 1, dh), ("w", 2, dw)):
        got = grad.to(F64).reshape(-1)
        for i in range(got.numel()):
            sides = []
            for sign in (1, -1):
                args = [x.clone(), r.clone(), w.clone()]
                args[arg].view(-1)[i] += sign * step
                sides.append(value(*args))
            want = (sides[0] - sides[1]) / (2 * step)
            # a difference's own error: the third derivative's step^2 and roundings of 2^-53 over the step; the call's: fp32
            assert abs(float(got[i]) - want) < 1e-4 * (1 + abs(want)), (what, i)


# ---------------------------------------------------------------------------- gated feed-forward block
SIZES = [(1, 1, 1), (1, 64, 64), (1, 2048, 640), (2, 8, 200), (3, 7, 5), (16, 1032, 72), (17, 65, 33), (31, 320, 1024),
         (33, 64, 128), (48, 72, 200), (5, 130, 4104), (4, 65, 9000), (9, 1500, 90), (6, 5001, 40), (64, 2048, 512), (129, 255, 130), (130, 128, 129), (257, 255, 1013), (300, 512, 384), (520, 1024, 640),
         (700, 40, 1500), (2050, 136, 2056), (1500, 704, 1400),
         # a moderate number of fp32 rows whose weights are read in place
         (17, 1029, 8200), (24, 8193, 1027), (33, 4099, 1032), (64, 2051, 4099), (65, 1001, 4203), (129, 16390, 257), (130, 257, 16500),
         (300, 1300, 1250), (512, 8200, 513)]
TYPES = [("f32", 16), ("bf16", 16), ("bf16", 8), ("f32", 8)]


def ffn_inputs(cuda, rows, width, hidden, dt, bits):
    g = gen(cuda, rows, width, hidden)
    scale = None
    X = rand(g, (rows, width), F32)
    if bits == 8:
        scale = torch.exp2(torch.ceil(torch.log2(X.abs().amax(1) / 448)))
        X = (X / scale[:, None]).to(E4M3)
    else:
        X = X.to(DT[dt])
    Wg, Wu = rand(g, (hidden, width), DT[dt], width ** -0.5), rand(g, (hidden, width), DT[dt], width ** -0.5)
    Wd, dY = rand(g, (width, hidden), DT[dt], hidden ** -0.5), rand(g, (rows, width), DT[dt])
    return X, scale, Wg, Wu, Wd, dY


@pytest.mark.parametrize("dt,bits", TYPES)
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_feed_forward(cuda, rows, width, hidden, dt, bits):
    import rank_orthonormalized_optimizer_amd as dion
    t = DT[dt]
    X, scale, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, bits)
    act = "silu" if rows % 2 else "gelu"
    want = Ffn(X, Wg, Wu, Wd, act, scale)
    Y, gate, up = Guarded((rows, width), t, cuda), Guarded((rows, hidden), t, cuda), Guarded((rows, hidden), t, cuda)
    ws = dirty(dion.gated_ffn_workspace_for(rows, width, hidden, cuda, t, x_dtype=X.dtype))
    assert dion.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale, gate=gate.t, up=up.t, out=Y.t, workspace=ws) is Y.t
    h = half_step(t)
    for name, got in (("gate", gate), ("up", up)):
        v, e = getattr(want, name), getattr(want, name + "_bound")
        # (a value next to a border of the form may be kept on its coarser side)
        step = torch.maximum(torch.maximum(keep_step(v, t), keep_step(v.abs() + e, t)), keep_step((v.abs() - e).clamp(min=0), t))
        close(kept(got.check()), v, e + step, name)
    close(Y.check(), want.Y, want.Y_bound + h * (want.Y.abs() + want.Y_bound), "Y")
    assert torch.equal(dion.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale), Y.t)   # nothing kept, its own workspace


@pytest.mark.parametrize("dt,bits", TYPES)
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_feed_forward_gradients(cuda, rows, width, hidden, dt, bits):
    import rank_orthonormalized_optimizer_amd as dion
    t = DT[dt]
    X, scale, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, bits)
    act = "gelu" if rows % 2 else "silu"
    names = ("dX", "dWg", "dWu", "dWd")
    for saved, wt, accumulate in ((True, t, False), (False, F32, True)):
        gate = up = None
        if saved:
            first = Ffn(X, Wg, Wu, Wd, act, scale)
            gate, up = keep(first.gate, t), keep(first.up, t)
        shapes = {"dX": (rows, width), "dWg": (hidden, width), "dWu": (hidden, width), "dWd": (width, hidden)}
        out = {k: Guarded(s, t if k == "dX" else wt, cuda) for k, s in shapes.items()}
        old = None
        if accumulate:
            for k in names[1:]:
                out[k].t.copy_(rand(gen(cuda, 3, rows), shapes[k], F32))
            old = {k: out[k].t.clone() for k in names[1:]}
        want = Ffn(X, Wg, Wu, Wd, act, scale, dY, gate, up, old)
        ws = dirty(dion.gated_ffn_workspace_for(rows, width, hidden, cuda, t, x_dtype=X.dtype, for_grad=True, saved=saved))
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, gate, up, *(out[k].t for k in names), act=act, scale=scale,
                             accumulate=accumulate, workspace=ws)
        for k in names:
            w, e = getattr(want, k), getattr(want, k + "_bound")
            h = half_step(t if k == "dX" else wt)
            close(out[k].check(), w, e + h * (w.abs() + e), f"{k} (saved {saved})")
        if saved:   # one output at a time (whose reductions may be cut elsewhere)
            for some in (("dX",), ("dWg", "dWu"), ("dWd",)):
                alone = {k: Guarded(shapes[k], t, cuda) for k in some}
                dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, gate, up, act=act, scale=scale, **{k: v.t for k, v in alone.items()})
                for k, v in alone.items():
                    w, e = getattr(want, k), getattr(want, k + "_bound")
                    close(v.check(), w, e + half_step(t) * (w.abs() + e), f"{k} alone")


def test_kept_form(cuda):
    """One product with ones passes any value on to gate: borders, ties, subnormal numbers and both signs come back as the
    form says."""
    import rank_orthonormalized_optimizer_amd as dion
    v = torch.tensor([0.0, 1.0, 1 + 2 ** -7, 2.0 ** -8, 2.0 ** -8 * (1 - 2 ** -8), 255.0, 256.0, 254.0, 3e38, 1e-38, 2.0 ** -130, 0.1,
                      100.5, 1e-3, 1e4], device=cuda)
    v = torch.cat([v, -v]).to(BF16)   # bf16 operands pass on unrounded
    X = torch.zeros(v.numel(), 64, device=cuda, dtype=BF16)
    X[:, 0] = v
    Wg = torch.zeros(8, 64, device=cuda, dtype=BF16)
    Wg[:, 0] = 1
    gate, up = torch.empty(v.numel(), 8, device=cuda, dtype=BF16), torch.empty(v.numel(), 8, device=cuda, dtype=BF16)
    dion.gated_ffn_(X, Wg, Wg, Wg.t().contiguous(), gate=gate, up=up)
    normal = v.abs().float() >= 2.0 ** -126   # (the matrix cores may count smaller ones as zero)
    want = keep(v, BF16)
    assert torch.equal(gate.view(torch.int16)[normal], want.view(torch.int16)[normal][:, None].expand(-1, 8))
    assert torch.equal(gate.view(torch.int16), up.view(torch.int16))
    assert ((kept(want) - v.to(F64)).abs() <= keep_step(v.to(F64), BF16)).all()


def test_feed_forward_without_rows(cuda):
    import rank_orthonormalized_optimizer_amd as dion
    for t in (F32, BF16):
        X, Wg, Wu, Wd = (torch.randn(s, device=cuda).to(t) for s in ((0, 24), (40, 24), (40, 24), (24, 40)))
        assert dion.gated_ffn_(X, Wg, Wu, Wd).shape == (0, 24)
        dW = [torch.full(s, float("nan"), device=cuda, dtype=t) for s in ((40, 24), (40, 24), (24, 40))]
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, X, None, None, torch.empty_like(X), *dW)
        assert all((g == 0).all() for g in dW)
        dW[0].fill_(3.0)
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, X, None, None, None, *dW, accumulate=True)
        assert (dW[0] == 3).all() and (dW[1] == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t", [F32, BF16])
def test_feed_forward_far_out(cuda, t, act):
    """Projections of thousands, where the activation is its argument or zero: no NaN, and the bound holds."""
    import rank_orthonormalized_optimizer_amd as dion
    g = gen(cuda, 6)
    rows, width, hidden = 40, 72, 136
    X, Wg = rand(g, (rows, width), t, 100.0), rand(g, (hidden, width), t, 10.0)
    Wu, Wd, dY = rand(g, (hidden, width), t), rand(g, (width, hidden), t), rand(g, (rows, width), t)
    want = Ffn(X, Wg, Wu, Wd, act)
    Y = dion.gated_ffn_(X, Wg, Wu, Wd, act=act)
    close(Y, want.Y, want.Y_bound + half_step(t) * (want.Y.abs() + want.Y_bound), "Y")
    out = [torch.empty_like(v) for v in (X, Wg, Wu, Wd)]
    dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, None, None, *out, act=act)
    want = Ffn(X, Wg, Wu, Wd, act, dY=dY)
    for k, v in zip(("dX", "dWg", "dWu", "dWd"), out):
        w, e = getattr(want, k), getattr(want, k + "_bound")
        close(v, w, e + half_step(t) * (w.abs() + e), k)


PATHS = [("f32", 3, 100, 4000), ("f32", 20, 1030, 8200), ("f32", 40, 2100, 2003), ("f32", 40, 70, 300), ("f32", 100, 1100, 4000),
         ("f32", 200, 255, 1013), ("f32", 520, 300, 500), ("bf16", 3, 100, 4000), ("bf16", 100, 320, 1000), ("bf16", 257, 255, 130)]


@pytest.mark.parametrize("dt,rows,width,hidden", PATHS)
def test_feed_forward_in_graphs(cuda, dt, rows, width, hidden):
    """Every way through the block, captured twice over one workspace: each replay as the eager call, bit for bit, whatever the
    workspace holds before."""
    import rank_orthonormalized_optimizer_amd as dion
    t = DT[dt]
    X, _, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, 16)
    ws = dirty(max((dion.gated_ffn_workspace_for(rows, width, hidden, cuda, t, for_grad=g, saved=s) for g, s in
                    ((False, True), (True, True), (True, False))), key=lambda w: w.numel()))
    gate, up = (torch.empty(rows, hidden, device=cuda, dtype=t) for _ in range(2))
    Y = torch.empty_like(X)
    out = [torch.empty_like(v) for v in (X, Wg, Wu, Wd)]
    again = [torch.empty_like(v) for v in out]

    def forward(ws=None):
        dion.gated_ffn_(X, Wg, Wu, Wd, gate=gate, up=up, out=Y, workspace=ws)

    def backward(ws=None):
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, gate, up, *out, workspace=ws)
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, None, None, *again, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward()
        backward()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (forward, backward):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f(ws)
    for i in range(3):
        X.copy_(X.roll(1, 0))
        dY.mul_(-1)
        dirty(ws)
        for g in graphs:
            g.replay()
        got = [v.clone() for v in (gate, up, Y, *out, *again)]
        forward()
        backward()
        for a, b in zip(got, (gate, up, Y, *out, *again)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dt,rows,width,hidden", PATHS)
def test_feed_forward_keeps_what_is_not_finite_apart(cuda, dt, rows, width, hidden):
    """A row that is not finite reaches its own row of Y and dX, a weight's row its own column of gate; everything else stays as
    it was, bit for bit."""
    import rank_orthonormalized_optimizer_amd as dion
    t = DT[dt]
    X, _, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, dt, 16)

    def run():
        gate, up = (torch.empty(rows, hidden, device=cuda, dtype=t) for _ in range(2))
        Y, dX = dion.gated_ffn_(X, Wg, Wu, Wd, gate=gate, up=up), torch.empty_like(X)
        dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, gate, up, dX)
        return gate, up, Y, dX
    clean = run()
    bad = rows - 2
    X[bad, width - 1], dY[bad, 0] = float("inf"), float("nan")
    rest = torch.arange(rows, device=cuda) != bad
    for name, a, b in zip(("gate", "up", "Y", "dX"), run(), clean):
        assert torch.equal(a[rest], b[rest]), name
    assert torch.isnan(run()[3][bad]).any()
    X[bad, width - 1], dY[bad, 0] = 0, 0
    clean = run()
    for j, c in ((1, 0), (hidden - 1, width - 1)):   # the ends of a row, whose neighbours are other rows
        Wg[j, c] = float("nan")
    gate, up, _, _ = run()
    other = torch.ones(hidden, dtype=torch.bool, device=cuda)
    other[1] = other[hidden - 1] = False
    assert torch.equal(gate[:, other], clean[0][:, other]) and torch.equal(up, clean[1])
    assert torch.isnan(kept(gate) if t == BF16 else gate)[:, ~other].all()
