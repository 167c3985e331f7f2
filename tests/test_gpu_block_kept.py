"""GPU tests of the form in which the feed-forward block's two projections are kept between its passes: gradients at any scale of
the weights are at least as exact as from projections kept in bf16."""
import pytest
import torch

from tests.block_reference import F64, Ffn, Guarded, activation, close, half_step
from tests.test_gpu_block import ffn_inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def kept_even(t):
    """The values of a buffer in the even form of dion_block.h."""
    c = t.view(torch.int16).to(torch.int64) & 0xffff
    n = c & 0x3fff
    e = torch.where(c >> 14 & 1 == 1, (n >> 10) - 8, torch.where(n >> 7 < 72, (n >> 7) - 80, (n >> 7) - 64))
    f = torch.where(c >> 14 & 1 == 1, (n & 1023) / 1024.0, (n & 127) / 128.0).to(F64)
    v = torch.exp2(e.to(F64)) * (1 + f)
    v = torch.where(c & 0x7fff == 0, 0.0, torch.where(c & 0x7fff == 0x3fff, torch.nan, v))
    return torch.where(c >> 15 == 1, -v, v)


def gradients(X, Wg, Wu, Wd, dY, act, a, b, part):
    """The block's gradients in 64 bits from a and b, with da, db and u rounded by ``part``."""
    x, wg, wu, wd, dy = (t.to(F64) for t in (X, Wg, Wu, Wd, dY))
    v, slope, _ = activation(act, a)
    du = dy @ wd
    da, db, u = part(du * b * slope), part(du * v), part(v * b)
    return {"dX": da @ wg + db @ wu, "dWg": da.t() @ x, "dWu": db.t() @ x, "dWd": dy.t() @ u}


def same(t):
    return t


def to_bf16(t):
    return t.to(BF16).to(F64)


def case(cuda, rows, size):
    g = torch.Generator(device=cuda).manual_seed(rows * 1000 + int(size) + 11)
    width, hidden = 256, 384

    def rnd(*s, std=1.0):
        return (torch.randn(*s, generator=g, device=cuda) * std).to(BF16)
    X, dY = rnd(rows, width), rnd(rows, width)
    Wg, Wu = rnd(hidden, width, std=2.0 ** size / 16), rnd(hidden, width, std=2.0 ** size / 16)
    return X, Wg, Wu, rnd(width, hidden, std=1 / 16), dY


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", [-40, -10, -7, 0, 10])
@pytest.mark.parametrize("rows", [5, 12, 40, 300])
def test_gradients_are_as_exact_as_from_projections_kept_in_bf16(cuda, rows, size, act):
    """Projections of about 2^size.  The errors (of norms, against 64 bits) are compared with those of a and b rounded to bf16 and
    da, db and u to what they multiply as, all else exact: norms of at least 5 x 256 errors, which differ by chance by
    1 / sqrt(2 x 1280) = 2%, so 1.15 is seven times that; half a bit less of a and b would make it 1.5."""
    import rank_orthonormalized_optimizer_amd as dion
    X, Wg, Wu, Wd, dY = case(cuda, rows, size)
    a, b = X.to(F64) @ Wg.to(F64).t(), X.to(F64) @ Wu.to(F64).t()
    part = same if rows <= 16 else to_bf16   # (few rows: two parts)
    exact = gradients(X, Wg, Wu, Wd, dY, act, a, b, same)
    rounded = gradients(X, Wg, Wu, Wd, dY, act, to_bf16(a), to_bf16(b), part)
    rounded["dX"] = to_bf16(rounded["dX"])
    for keep in (True, False):
        opt = dion.MixedDion([Wg.clone(), Wu.clone(), Wd.clone()])
        _, kept = opt.feed_forward((0, 1, 2), X, act=act, keep=keep)
        got = dict(zip(("dWg", "dWu", "dWd"), (None,) * 3))
        got["dX"] = opt.feed_forward_grad((0, 1, 2), X, dY, kept, act=act)
        got["dWg"], got["dWu"], got["dWd"] = (opt.gathered[i] for i in range(3))
        for k, want in exact.items():
            off, most = float((got[k].to(F64) - want).norm() / want.norm()), float((rounded[k] - want).norm() / want.norm())
            assert off <= 1.15 * most, (k, keep, off, most)


def test_the_even_form(cuda):
    """One product with ones passes any value on to gate: borders, ties and both signs come back as the form says."""
    import rank_orthonormalized_optimizer_amd as dion
    below = 2.0 ** -8
    codes = {0.0: 0, 1.0: 0x4000 | 8 << 10, below: 0x4000, below * (1 - 2 ** -8): 71 << 7 | 127, 255.0: 0x4000 | 15 << 10 | 1016,
             256.0: 72 << 7, 258.0: 72 << 7 | 1, 3e38: 0x3fff, 2.0 ** 63 * (1 + 126 / 128): 0x3ffe, 2.0 ** 63 * (1 + 127 / 128): 0x3fff,
             2.0 ** 64: 0x3fff, float("inf"): 0x3fff, float("nan"): 0x3fff, 2.0 ** -80: 0, 2.0 ** -80 * (1 + 2 ** -7): 1, 2.0 ** -81: 0,
             2.0 ** -79: 1 << 7, 1e-38: 0, 1 + 2 ** -7: 0x4000 | 8 << 10 | 8, 2.0 ** -9 * 1.5: 71 << 7 | 64}
    # sums of two products, which bf16 cannot hold: ties, and what rounds up across a border
    sums = {(1.0, 2.0 ** -11): 0x4000 | 8 << 10 | 1, (1.0, 2.0 ** -11 * (1 - 2 ** -8)): 0x4000 | 8 << 10, (256.0, 1.0): 72 << 7 | 1,
            (256.0, 0.99609375): 72 << 7, (below * (1 - 2 ** -8), below * 2.0 ** -9): 0x4000, (below, -below * 2.0 ** -12): 0x4000,
            (256.0, -0.0625): 72 << 7, (256.0, -0.0634765625): 0x4000 | 15 << 10 | 1023, (512.0, -1.0): 73 << 7,
            (512.0, -1.0078125): 72 << 7 | 127}
    rows = [(v, 0.0, c) for v, c in codes.items()] + [(a, b, c) for (a, b), c in sums.items()]
    rows += [(-a, -b, c | 0x8000) for a, b, c in rows if a == a]
    X = torch.zeros(len(rows), 64, device=cuda, dtype=BF16)
    X[:, 0], X[:, 1] = (torch.tensor([r[i] for r in rows], device=cuda).to(BF16) for i in (0, 1))
    Wg = torch.zeros(8, 64, device=cuda, dtype=BF16)
    Wg[:, :2] = 1
    want = torch.tensor([r[2] for r in rows], device=cuda)[:, None].expand(-1, 8)
    for n in (len(rows), 7):   # (few rows go another way)
        for at in range(0, len(rows) - n + 1, n):
            gate, up = (torch.empty(n, 8, device=cuda, dtype=torch.int16) for _ in range(2))
            dion.gated_ffn_(X[at:at + n].clone(), Wg, Wg, Wg.t().contiguous(), gate=gate, up=up)
            wrong = (gate.to(torch.int64) & 0x7fff) != (want[at:at + n] & 0x7fff)
            assert not wrong.any(), [rows[at + i] for i in wrong.any(1).nonzero()[:, 0].tolist()]
            # (a NaN has any sign; -0 x 1 + 0 is 0, and the matrix cores may count subnormal numbers as zero)
            signed = (want[at:at + n] & 0x7fff != 0x3fff) & (X[at:at + n, :1].float().abs() >= 2.0 ** -126)
            assert ((gate.to(torch.int64) & 0xffff)[signed] == want[at:at + n][signed]).all()
            assert torch.equal(gate, up)


@pytest.mark.parametrize("rows,width,hidden,bits", [(1, 64, 64, 16), (3, 7, 5, 8), (8, 2048, 640, 16), (9, 320, 1024, 16), (16, 64, 1001, 16),
                                                    (40, 255, 130, 8), (64, 128, 200, 16), (257, 255, 1013, 16), (700, 40, 1500, 8),
                                                    (2050, 136, 2056, 16)])
def test_even_form_between_the_passes(cuda, rows, width, hidden, bits):
    """gate and up in the even form: values within its step of the projections, and gradients of what they stand for."""
    import rank_orthonormalized_optimizer_amd as dion
    X, scale, Wg, Wu, Wd, dY = ffn_inputs(cuda, rows, width, hidden, "bf16", bits)
    act = "gelu" if rows % 2 else "silu"
    want = Ffn(X, Wg, Wu, Wd, act, scale)
    gate, up = (Guarded((rows, hidden), torch.int16, cuda) for _ in range(2))
    Y = dion.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale, gate=gate.t, up=up.t)
    assert torch.equal(Y, dion.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale))
    for name, got in (("gate", gate), ("up", up)):
        v, e = getattr(want, name), getattr(want, name + "_bound")
        fine = (v.abs() - e >= 2.0 ** -8) & (v.abs() + e < 2.0 ** 8)   # (a value next to the window's border: either side's step)
        close(kept_even(got.check()), v, e + torch.where(fine, 2.0 ** -11, 2.0 ** -8) * (v.abs() + e) + 2.0 ** -80, name)
    # the reference takes the values as given: from fp32 weights' buffers, which are read as they are
    a, b = kept_even(gate.t).float(), kept_even(up.t).float()
    out = {k: Guarded(v.shape, BF16, cuda) for k, v in (("dX", Y), ("dWg", Wg), ("dWu", Wu), ("dWd", Wd))}
    dion.gated_ffn_grad_(X, Wg, Wu, Wd, dY, gate.t, up.t, *(g.t for g in out.values()), act=act, scale=scale)
    want = Ffn(X, Wg, Wu, Wd, act, scale, dY, a, b)
    for k, g in out.items():
        w, e = getattr(want, k), getattr(want, k + "_bound")
        close(g.check(), w, e + half_step(BF16) * (w.abs() + e), k)
