"""The residual blocks' operators' definitions in 64 bits (torch, any device) and the error bounds their
32-bit kernels are held to, element by element.

u = 2^-24 is half a step of fp32; a rounding to type t costs at most finfo(t).eps / 2 relative.

h       x's scale, its product and the addition: 3 u (|x| / (1 - p) + |residual|), then the output's rounding.
rstd    the squares' sum: 2 |h| e_h + u h^2 each, and sums of at most 64 + 6 + 16 terms on a path: relative
        2 sum(|h| e_h) / sum(h^2) + 88 u, halved by the root, and four roundings: c_r.
y       |y| (c_r + 2 u) + e_h rstd |w|, then the output's rounding.  In 8 bits: formed in fp64, equal.
dh      mean(g n): products and sums of at most 64 + 22 terms on a path, 90 u mean(|g n|); then
        rstd (4 u |g| + |n| e_mean + 6 u |n mean|) + 3 u |dh| + u |dsum|.  dx: two more roundings, times 1 / (1 - p).
dw      a sum of rows products: at most (rows + 40) u sum(|dY n|).
a, b    K products of 16-bit parts added in fp32: nseg K additions, doubled for the matrix core's own
        rounding, and 12 u for fp32 operands' dropped terms: (2 nseg K + 12) u sum |x| |w| (nseg 6 covers three
        products, and single ones in fp32).  Two fp16 parts of a row scaled to [2^13, 2^14) leave 2^-39 of the row's largest
        besides, where the low part is subnormal: 2^-38 (max|x| sum|w| + max|w| sum|x|).
du      the same, but Wd's rows k run along the reduction: with m_k = max |Wd_k|, 2^-38 (max_k (|dY_k| m_k)
        sum_k |Wd_kc| / m_k + sum_k |dY_k| m_k).
act     |act'| <= 1.2 and |act''| <= 1.2.  The sigmoid's argument z has a rounding of |z| 2 u (gelu's
        polynomial 4 u |z|), which is relative in its exponential, and eight u follow: relative 8 (|z| + 1) u
        of act, and of each of the two terms of act'.
the rest  by |ab - a'b'| <= (|a| + e_a)(|b| + e_b) - |a b|, the rounding of u, da and db to the parts they
        multiply as, and the products' additions as above.
"""
import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


class Guarded:
    """A tensor inside a larger buffer whose borders hold a pattern; filled with NaN, or 0xff bytes."""
    EDGE = 64

    def __init__(self, shape, dtype, device):
        n, edge = math.prod(shape), self.EDGE
        size = torch.empty(0, dtype=dtype).element_size()
        self.whole = torch.full(((n + 2 * edge + 16) * size,), 0x5a, dtype=torch.uint8, device=device)
        self.lo, self.hi = edge * size, (edge + n) * size
        inside = self.whole[self.lo:self.hi]
        inside.fill_(0xff)
        self.t = inside.view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        assert (self.whole[:self.lo] == 0x5a).all() and (self.whole[self.hi:] == 0x5a).all(), "written outside"
        return self.t


def dirty(ws):
    return ws.fill_(255)


def close(got, want, bound, what):
    got = got.to(F64).reshape(want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN where none belongs, or none where one does"
    fine = ~torch.isnan(want)
    worst = ((got - want).abs() - bound)[fine]
    assert worst.numel() == 0 or float(worst.max()) <= 0, \
        f"{what}: {float((got - want).abs()[fine].max())} off, {int((worst > 0).sum())} of {worst.numel()} values over their bound"


def mask(n: int, p: float, seed: int, site: int, device="cpu", start: int = 0):
    """Philox4x32-10's words of the n elements from ``start`` (a multiple of four) against p, products from 16-bit halves."""
    m32 = 0xffffffff

    def mul(a, m):
        lo = (a & 0xffff) * (m & 0xffff)
        mid = (a >> 16) * (m & 0xffff) + (lo >> 16)
        mid2 = (a & 0xffff) * (m >> 16) + (mid & 0xffff)
        return (a >> 16) * (m >> 16) + (mid >> 16) + (mid2 >> 16), (mid2 & 0xffff) << 16 | lo & 0xffff
    i = torch.arange(start // 4, (start + n + 3) // 4, device=device)
    key, site = seed % 2 ** 64, site % 2 ** 64
    c = [i & m32, i >> 32, torch.full_like(i, site & m32), torch.full_like(i, site >> 32)]
    k0, k1 = key & m32, key >> 32
    for _ in range(10):
        h0, l0 = mul(c[0], 0xD2511F53)
        h1, l1 = mul(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return (torch.stack(c, 1).reshape(-1)[:n] >= min(round(p * 2 ** 32), m32))


def kept(t):
    """The values of a gate or up buffer: fp32, or a bf16 buffer's bits in the 16-bit form of dion_block.h."""
    if t.dtype == torch.float32:
        return t.to(F64)
    c = t.view(torch.int16).to(torch.int64) & 0xffff
    e, f = torch.where(c >> 14 & 1 == 1, (c >> 10 & 15) - 8, (c >> 6 & 255) - 127), \
        torch.where(c >> 14 & 1 == 1, (c & 1023) / 1024.0, (c & 63) / 64.0).to(F64)
    v = torch.exp2(e.to(F64)) * (1 + f)
    v = torch.where(e == -127, torch.exp2(torch.full_like(v, -126)) * f, v)
    v = torch.where(e == 128, torch.where(f == 0, math.inf, math.nan).to(F64), v)
    return torch.where(c >> 15 == 1, -v, v)


def keep_step(v, dtype):
    """The most that keeping v rounds away."""
    if dtype == torch.float32:
        return U * v.abs()
    fine = (v.abs() >= 2.0 ** -8) & (v.abs() < 2.0 ** 8)
    return torch.where(fine, 2.0 ** -11, 2.0 ** -7) * v.abs() + 2.0 ** -132


def keep(v, dtype):
    """v in the form in which gate and up are kept."""
    if dtype == torch.float32:
        return v.float()
    bits = v.float().contiguous().view(torch.int32).to(torch.int64) & 0xffffffff
    m = bits & 0x7fffffff
    fine = ((m + 0x1000) >> 13) - (119 << 10)
    far = ((m + 0x10000) >> 17).clamp(max=0x3fff)
    c = torch.where((fine >= 0) & (fine < 0x4000), fine | 0x4000, far) | bits >> 16 & 0x8000
    return torch.where(c >= 0x8000, c - 0x10000, c).to(torch.int16).view(torch.bfloat16)


class Norm:
    """h, rstd, y and their bounds (before the outputs' rounding)."""

    def __init__(self, x, w, eps, residual=None, p=0.0, keep=None):
        d = x.shape[-1]
        x64, s = x.to(F64).reshape(-1, d), 1.0 / (1.0 - p)
        if keep is not None:
            x64 = torch.where(keep.reshape(-1, d), x64, 0.0)
        r64 = torch.zeros_like(x64) if residual is None else residual.to(F64).reshape(-1, d)
        self.h = x64 * s + r64
        self.h_bound = 3 * U * (x64.abs() * s + r64.abs())
        total = (self.h * self.h).sum(1)
        self.rstd = (total / d + eps) ** -0.5
        c = (self.h.abs() * self.h_bound).sum(1) / (total + d * eps) + 48 * U
        c = torch.nan_to_num(c, nan=48 * U)
        self.rstd_bound = c * self.rstd
        w64 = w.to(F64)
        self.y = self.h * self.rstd[:, None] * w64
        self.y_bound = self.y.abs() * (c[:, None] + 2 * U) + self.h_bound * self.rstd[:, None] * w64.abs()

    def eight(self):
        """(values, scale): y in e4m3 with the least power of two that holds the row."""
        finite = torch.where(torch.isfinite(self.y), self.y.abs(), 0.0)
        top = finite.amax(1)
        m, e = torch.frexp(top)
        scale = torch.where(top > 0, torch.exp2((e - 9 + (m > 0.875)).to(F64)), 1.0)
        v = self.y / scale[:, None]
        _, e = torch.frexp(v.abs().clamp(min=2.0 ** -6))
        step = torch.exp2((e - 4).to(F64))
        v = torch.round(v / step) * step
        return torch.where(torch.isfinite(v), v, math.nan), scale


class NormGrad:
    def __init__(self, dY, h, w, rstd, dsum=None, p=0.0, keep=None, old=None):
        d = h.shape[-1]
        dy, h64, w64, r = dY.to(F64).reshape(-1, d), h.to(F64).reshape(-1, d), w.to(F64), rstd.to(F64).reshape(-1, 1)
        s64 = torch.zeros_like(dy) if dsum is None else dsum.to(F64).reshape(-1, d)
        n, g = h64 * r, dy * w64
        mean = (g * n).mean(1, keepdim=True)
        e_mean = 90 * U * (g * n).abs().mean(1, keepdim=True)
        self.dh = r * (g - n * mean) + s64
        self.dh_bound = r * (4 * U * g.abs() + n.abs() * e_mean + 6 * U * (n * mean).abs()) + 3 * U * self.dh.abs() + U * s64.abs()
        k = torch.ones_like(dy) if keep is None else keep.reshape(-1, d).to(F64)
        self.dx = self.dh * k / (1 - p)
        self.dx_bound = k / (1 - p) * (self.dh_bound + 2 * U * self.dh.abs())
        o64 = 0.0 if old is None else old.to(F64)
        self.dw = (dy * n).sum(0) + o64
        self.dw_bound = (dy.shape[0] + 40) * U * (dy * n).abs().sum(0) + (0.0 if old is None else 2 * U * o64.abs())


def activation(act, a):
    """act(a), its derivative, and the size of the sigmoid's argument."""
    if act == "silu":
        r = torch.sigmoid(a)
        return a * r, r + a * r * (1 - r), a.abs()
    c = 2 * math.sqrt(2 / math.pi)
    z = c * (a + 0.044715 * a ** 3)
    r = torch.sigmoid(z)
    return a * r, r + a * r * (1 - r) * c * (1 + 0.134145 * a * a), 2 * z.abs()


def _both(a, ea, b, eb):
    return (a.abs() + ea) * (b.abs() + eb) - (a * b).abs()


class Ffn:
    """Everything of one feed-forward block in 64 bits, with bounds before the outputs' rounding.  ``gate`` and ``up``: as
    stored, taken as given; else formed, and rounded as they would be kept where ``grad``."""

    def __init__(self, X, Wg, Wu, Wd, act, scale=None, dY=None, gate=None, up=None, old=None):
        t = Wg.dtype
        x, wg, wu, wd = (v.to(F64) for v in (X.reshape(-1, X.shape[-1]), Wg, Wu, Wd))
        if scale is not None:
            x = x * scale.to(F64).reshape(-1, 1)
        T, d, f = x.shape[0], x.shape[1], wg.shape[0]
        bf16 = t == torch.bfloat16
        nseg, part = (1, half_step(t)) if bf16 else (6, U)   # products of parts, and what is left out of u, da and db
        if bf16 and T <= (64 if dY is None else 16):   # two parts: the second one's rounding is left
            nseg, part = 2, half_step(t) ** 2

        def grow(k):
            return (2 * nseg * k + 12) * U
        a, b = x @ wg.t(), x @ wu.t()
        ea, eb = grow(d) * (x.abs() @ wg.abs().t()), grow(d) * (x.abs() @ wu.abs().t())
        if not bf16:
            for e, w in ((ea, wg), (eb, wu)):
                e += 2.0 ** -38 * (x.abs().amax(1)[:, None] * w.abs().sum(1) + x.abs().sum(1)[:, None] * w.abs().amax(1))
        self.gate, self.up, self.gate_bound, self.up_bound = a, b, ea, eb
        if dY is not None:
            if gate is not None:
                a, b = kept(gate).reshape(T, f), kept(up).reshape(T, f)
                ea, eb = torch.zeros_like(a), torch.zeros_like(b)
            else:
                # (a value next to a border of the form may fall on its coarser side)
                ea, eb = ea + torch.maximum(keep_step(a, t), keep_step(a.abs() + ea, t)), eb + torch.maximum(keep_step(b, t), keep_step(b.abs() + eb, t))
        v, slope, z = activation(act, a)
        rel = 8 * (z + 1) * U
        ev = 1.2 * ea + rel * v.abs()
        u = v * b
        eu = _both(v, ev, b, eb)
        eu = eu + (part + U) * (u.abs() + eu)
        self.Y = u @ wd.t()
        self.Y_bound = eu @ wd.abs().t() + grow(f) * ((u.abs() + eu) @ wd.abs().t())
        if dY is None:
            return
        dy = dY.to(F64).reshape(T, d)
        du = dy @ wd
        edu = grow(d) * (dy.abs() @ wd.abs())
        if not bf16:
            m = wd.abs().amax(1).clamp(min=2.0 ** -87)
            edu += 2.0 ** -38 * ((dy.abs() * m).amax(1)[:, None] * (wd.abs() / m[:, None]).sum(0) + (dy.abs() @ m)[:, None])
        es = 1.2 * ea + rel * (slope.abs() + 2 + v.abs())
        e1 = _both(du, edu, b, eb)
        da, db = du * b * slope, du * v
        eda, edb = _both(du * b, e1, slope, es), _both(du, edu, v, ev)
        eda, edb = eda + (part + 2 * U) * (da.abs() + eda), edb + (part + U) * (db.abs() + edb)
        self.dX = da @ wg + db @ wu
        self.dX_bound = eda @ wg.abs() + edb @ wu.abs() + grow(2 * f) * ((da.abs() + eda) @ wg.abs() + (db.abs() + edb) @ wu.abs())
        outs = {"dWg": (da, eda, x), "dWu": (db, edb, x), "dWd": None}
        for k in outs:
            if k == "dWd":
                g = dy.t() @ u
                e = dy.abs().t() @ eu + grow(T) * (dy.abs().t() @ (u.abs() + eu))
            else:
                m, em, right = outs[k]
                g = m.t() @ right
                e = em.t() @ right.abs() + grow(T) * ((m.abs() + em).t() @ right.abs())
            if old is not None:
                g = g + old[k].to(F64)
                e = e + 2 * U * (old[k].to(F64).abs() + g.abs())
            setattr(self, k, g)
            setattr(self, k + "_bound", e)
