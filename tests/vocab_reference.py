"""The vocabulary operators' definitions in 64 bits (torch, any device) and the error bounds their
32-bit kernels are held to, element by element.

u = 2^-24 is half a step of fp32; a rounding to type t costs at most finfo(t).eps / 2 relative.

lookup   one fp32 multiplication and one rounding: equal bit for bit to the same in torch.
table    a row of c tokens: c - 1 additions, the scale and an addition to what was there, each one
         rounding of a partial result that is at most |scale| sum |dY| + |old|: (c + 4) u of that,
         then the output's rounding.
logits   K products of 16-bit parts added in fp32: at most nseg K additions, doubled for the matrix
         core's own rounding (it need not be to nearest), of values at most sum_k |h||w|: 2 nseg K u.
         fp32 operands go as two fp16 parts of a row scaled to [2^13, 2^14): each part's rounding
         leaves 2^-23 of the element or, where the low part is subnormal, 2^-39 of the row's largest;
         the dropped l l product is below 2^-22: (2 + 2 + 4) u sum_k |h||w| and
         2^-38 (max|h| sum|w| + max|w| sum|h|).  gamma_z = (2 nseg K + 12) u.
lse      the largest logit error, plus sums of at most V exponentials (added in a tree of at most
         96 + V / 64 steps per path), four u for each exponential, and two roundings of |lse|.
D        p (error of the logit and lse, and four u), then grad's multiplication and the rounding of
         D to its parts: 2^-8 for one bf16 part, u for three.
dH, dW   those errors through the products, and the products' own additions as for the logits.
         dH of fp32 operands may come from two fp16 parts of D times W's inverse row scales (at most `top`) and of the
         scaled rows of W: 2^-23 of each factor and 2^-22 for the dropped l l, 8 u in all, and where a low part of D is
         subnormal 2^-39 top |W / inverse|, at most 2^-38 max |W| per row of W (a power of two of grad's size outside).
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def table(ids, dY, vocab, scale, padding_id=-1, old=None):
    """(dW, bound before the output's rounding) for flat ids."""
    f64 = torch.float64
    d = dY.shape[-1]
    keep = (ids >= 0) & (ids < vocab) & (ids != padding_id)
    k = ids[keep].long()
    rows = dY.reshape(-1, d)[keep].to(f64) * scale
    zero = torch.zeros(vocab, d, dtype=f64, device=dY.device)
    old = zero if old is None else old.to(f64)
    out = old + zero.index_add(0, k, rows)
    size = old.abs() + zero.index_add(0, k, rows.abs())
    count = torch.zeros(vocab, dtype=f64, device=dY.device).index_add(0, k, torch.ones(k.numel(), dtype=f64, device=dY.device))
    return out, (count[:, None] + 4) * U * size


class Head:
    """Everything of one cross entropy call in 64 bits: loss, lse, and with ``grad`` dH and dW, with bounds."""

    def __init__(self, H, W, targets, ignore=-100, grad=None, dw_dtype=None, dw_old=None):
        f64, dev = torch.float64, H.device
        d, V = H.shape[-1], W.shape[0]
        h32 = H.reshape(-1, d)
        y = targets.reshape(-1).long()
        keep = y != ignore
        h = torch.where(keep[:, None], h32.to(f64), 0.0)   # an ignored row may hold anything
        w = W.to(f64)
        parts = 1 if H.dtype == torch.bfloat16 else 3
        dparts = 1 if parts == 1 and dw_dtype in (None, torch.bfloat16) else 3
        nz, nh = {1: (1, 1), 3: (3, 6)}[parts]             # part products of the logits and of dH
        z = h @ w.t()
        gz = (2 * nz * d + 12) * U
        size = (h.abs() @ w.abs().t()).amax(1)             # an error bound of every logit of the row, over gz
        if parts == 3:
            wa = w.abs()
            size = size + 2.0 ** -38 / gz * (h.abs().amax(1) * wa.sum(1).max() + wa.max() * h.abs().sum(1))
        self.lse = torch.where(keep, torch.logsumexp(z, 1), 0.0)
        inside = (y >= 0) & (y < V)
        rows = torch.arange(y.numel(), device=dev)
        zy = z[rows, y.clamp(0, V - 1)]
        self.loss = torch.where(keep, torch.where(inside, self.lse - zy, math.nan), 0.0)
        e_lse = gz * size + (96 + V / 64 + 4) * U + 2 * U * self.lse.abs()
        self.lse_bound = torch.where(keep, e_lse, 0.0)
        self.loss_bound = torch.where(keep, e_lse + gz * size + 4 * U * (z.amax(1).abs() + zy.abs()), 0.0)
        if grad is None:
            return
        g = (grad.to(f64).reshape(-1) if grad.numel() > 1 else grad.to(f64).reshape(1).expand(y.numel()))
        g = torch.where(keep, torch.where(inside, g, math.nan), 0.0)
        p = torch.exp(z - torch.where(keep, self.lse, math.inf)[:, None])
        D = p.clone()
        D[rows, y.clamp(0, V - 1)] -= inside.to(f64)
        D = torch.where(keep[:, None], D * g[:, None], 0.0)
        e1 = (gz * size + self.lse_bound + 6 * U)[:, None] * p * torch.where(keep, g, 0.0).abs()[:, None] + 2 * U * D.abs()

        def bound(rounding, a, nseg, length, left):
            e = e1 + rounding * D.abs()
            grow = (2 * nseg * length + 8) * U
            m = a.abs()
            return (e @ m + grow * (D.abs() @ m)) if left else (e.t() @ m + grow * (D.abs().t() @ m))

        rh = half_step(torch.bfloat16) if H.dtype == torch.bfloat16 else U
        rw = half_step(torch.bfloat16) if dparts == 1 else U
        self.dH = D @ w
        self.dH_bound = bound(rh, w, nh, V, True) + half_step(H.dtype) * self.dH.abs()
        if parts == 3:
            size_g = torch.where(keep, g, 0.0).abs()[:, None]
            self.dH_bound = self.dH_bound + 8 * U * (D.abs() @ w.abs()) + 2.0 ** -38 * V * w.abs().max() * size_g
        old = 0.0 if dw_old is None else dw_old.to(f64)
        self.dW = D.t() @ h + old
        self.dW_bound = bound(rw, h, {(1, 1): 1, (1, 3): 3, (3, 3): 6}[parts, dparts], y.numel(), False) \
            + half_step(dw_dtype or H.dtype) * 1.01 * self.dW.abs() + 2 * U * (0.0 if dw_old is None else old.abs())
