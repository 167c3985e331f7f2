"""torch-facing wrappers of include/dion_block.h: dropout, the root-mean-square norm with the residual's
addition, the gated feed-forward block, and their gradients (marshalling only, no arithmetic).

Tensors are contiguous and on one GPU; everything is enqueued on ``stream`` (default: torch's
current stream of that GPU) with no host sync.  Scratch and outputs that are not given are
allocated by torch on that stream.

No call records a graph for autograd: gradients are calls of their own.  Where autograd would expect
one, the forward calls refuse tensors that require a gradient: call them under ``torch.no_grad()`` or
on detached tensors.

Dropout's mask is never stored: it is a function of ``seed`` (an int64 tensor of one element on the
GPU, read when the kernel runs), ``site`` (a whole number that keeps the masks of different layers
apart) and an element's number, so that the gradient forms it again from the same three.
"""
from __future__ import annotations

import torch

from . import _lib
from .vocab import _DT, _given_scratch, _need, _On, _scratch

E4M3 = torch.float8_e4m3fn
_ACT = {"silu": _lib.SILU, "gelu": _lib.GELU}


def _no_graph(call: str, gradient: str, *tensors) -> None:
    if torch.is_grad_enabled():
        for name, t in tensors:
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{call} records no graph, but {name} requires a gradient: call it under torch.no_grad() "
                                 f"or detach {name}, and {gradient} for the gradient")


def _check(t, name: str, dtypes, device, shape) -> None:
    """_need on a tensor that is nearly always right: small calls take as long as their checks."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.device == device
            and t.is_contiguous()):
        _need(t, name, dtypes, device, shape)


def _ptr(t):
    return None if t is None else t.data_ptr()


_I64 = (torch.int64,)


def _seed(seed, p: float, device):
    if p == 0:   # it is not read
        return None
    if seed is None:
        raise ValueError("dropout needs a seed: an int64 GPU tensor of one element")
    _need(seed, "seed", _I64, device)
    if seed.numel() != 1:
        raise ValueError(f"seed has shape {tuple(seed.shape)}, expected one element")
    return seed.data_ptr()


def _space(like, nbytes: int) -> torch.Tensor:
    """_scratch on a tensor's GPU."""
    return like.new_empty(max(int(nbytes), 256), dtype=torch.uint8)


def _rows(x, name: str):
    """(rows, width) of a tensor [..., width]."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name} must have a width of at least 1, got shape {tuple(x.shape)}")
    return x.numel() // x.shape[-1], x.shape[-1]


def dropout_(x: torch.Tensor, p: float, seed: torch.Tensor | None = None, site: int = 0, *,
             residual: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``out = residual + keep * x / (1 - p)`` with a mask that is never stored (dion_dropout).

    x: float32 or bfloat16 of any shape; residual and out: x's shape, float32 or bfloat16 (default: the
    residual's type, else x's); out may be residual.  The gradient of x is the same call, without residual,
    on the output's gradient.
    """
    _no_graph("dropout_", "dropout_ of the output's gradient", ("x", x), ("residual", residual), ("out", out))
    _need(x, "x", _DT)
    device, shape = x.device, x.shape
    with _On(device, stream) as handle:
        if residual is not None:
            _check(residual, "residual", _DT, device, shape)
        if out is None:
            out = torch.empty_like(x if residual is None else residual)
        else:
            _check(out, "out", _DT if residual is None else (residual.dtype,), device, shape)
        st = _lib.load().dion_dropout(x.data_ptr(), _ptr(residual), out.data_ptr(), x.numel(), float(p),
                                      _seed(seed, p, device), int(site), _DT[x.dtype], _DT[out.dtype], handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_dropout")
    return out


_F32 = (torch.float32,)
_Q8 = (E4M3,)


def _norm(call, x, w, eps, residual, p, seed, site, h, y, scale, rstd, eight, stream):
    _no_graph(call, "rms_norm_grad_", ("x", x), ("w", w), ("residual", residual), ("h", h), ("out", y), ("scale", scale), ("rstd", rstd))
    _need(x, "x", _DT)
    device, shape = x.device, x.shape
    rows, width = _rows(x, "x")
    _check(w, "w", _DT, device, shape[-1:])
    with _On(device, stream) as handle:
        if residual is not None:
            _check(residual, "residual", _DT, device, shape)
        like = x if residual is None else residual   # the stream
        if h is not None:
            _check(h, "h", _DT if residual is None else (residual.dtype,), device, shape)
            like = h
        elif residual is not None or p != 0:
            h = torch.empty_like(like)
        if y is None:
            y = torch.empty_like(x, dtype=E4M3) if eight else torch.empty_like(x)
        else:
            _check(y, "out", _Q8 if eight else _DT, device, shape)
        per_row = shape[:-1]
        if eight:
            if scale is None:
                scale = x.new_empty(per_row, dtype=torch.float32)
            else:
                _check(scale, "scale", _F32, device, per_row)
        if rstd is None:
            rstd = x.new_empty(per_row, dtype=torch.float32)
        else:
            _check(rstd, "rstd", _F32, device, per_row)
        st = _lib.load().dion_rms_norm(x.data_ptr(), None if residual is None else residual.data_ptr(), w.data_ptr(),
                                       None if h is None else h.data_ptr(), y.data_ptr(),
                                       scale.data_ptr() if eight else None, rstd.data_ptr(), rows, width, eps, p,
                                       _seed(seed, p, device), site, _DT[x.dtype], _DT[like.dtype], _DT[w.dtype],
                                       _lib.E4M3 if eight else _DT[y.dtype], handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_rms_norm")
    return y, scale, x if h is None else h, rstd


def rms_norm_(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, *, residual: torch.Tensor | None = None, p: float = 0.0,
              seed: torch.Tensor | None = None, site: int = 0, h: torch.Tensor | None = None,
              out: torch.Tensor | None = None, rstd: torch.Tensor | None = None, stream=None):
    """``h = residual + dropout(x)`` and its root-mean-square norm ``y = h * rstd * w`` (dion_rms_norm).

    x: [..., width], w: [width], residual: x's shape, each float32 or bfloat16.  Returns (or fills) ``(y, h,
    rstd)``: y of x's shape and type (or out's), h of the residual's type (x itself where there is neither residual nor
    dropout and no ``h`` is given; ``h`` may be ``residual``), rstd float32 of x's shape without the width.
    """
    y, _, h, rstd = _norm("rms_norm_", x, w, eps, residual, p, seed, site, h, out, None, rstd, False, stream)
    return y, h, rstd


def rms_norm_8bit_(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, *, residual: torch.Tensor | None = None,
                   p: float = 0.0, seed: torch.Tensor | None = None, site: int = 0, h: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, scale: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                   stream=None):
    """rms_norm_ with y in 8 bits: returns (or fills) ``(q, scale, h, rstd)``, y standing as ``q * scale``.

    q: float8_e4m3fn; scale: float32 per row, the least power of two with max |y| <= 448 scale.  gated_ffn_ and
    gated_ffn_grad_ take the two; the gradient of the rounding is taken to be 1 (rms_norm_grad_ with y's gradient).
    """
    return _norm("rms_norm_8bit_", x, w, eps, residual, p, seed, site, h, out, scale, rstd, True, stream)


def rms_norm_grad_workspace_for(rows: int, width: int, device) -> torch.Tensor:
    """Scratch for one rms_norm_grad_ call of these sizes."""
    return _scratch(int(_lib.load().dion_rms_norm_grad_workspace_size(rows, width)), device)


def rms_norm_grad_(dY: torch.Tensor, h: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor, dw: torch.Tensor | None = None, *,
                   dsum: torch.Tensor | None = None, p: float = 0.0, seed: torch.Tensor | None = None, site: int = 0,
                   dh: torch.Tensor | None = None, dx: torch.Tensor | None = None, accumulate: bool = False,
                   workspace: torch.Tensor | None = None, stream=None):
    """Gradients of rms_norm_ and rms_norm_8bit_ (dion_rms_norm_grad); returns ``(dh, dx)`` and fills dw.

    dY: y's gradient, [..., width]; h, rstd: the forward call's; dsum: the gradient that reaches h by other ways, of
    h's type; dh: h's gradient, which is the residual's (may be dsum); dx: x's gradient, of dY's type, with the same p, seed and site.
    Without dropout dx is dh, unless a ``dx`` is given (where x has another type than the stream).  dw: [width] float32
    or bfloat16, written, or added to with ``accumulate``.
    """
    _need(dY, "dY", _DT)
    device, shape = dY.device, dY.shape
    rows, width = _rows(dY, "dY")
    _check(h, "h", _DT, device, shape)
    _check(w, "w", _DT, device, shape[-1:])
    _check(rstd, "rstd", _F32, device, shape[:-1])
    if dsum is not None:
        _check(dsum, "dsum", (h.dtype,), device, shape)
    if dw is not None:
        _check(dw, "dw", _DT, device, shape[-1:])
    with _On(device, stream) as handle:
        if dh is None:
            dh = torch.empty_like(h)
        else:
            _check(dh, "dh", (h.dtype,), device, shape)
        if dx is not None:
            _check(dx, "dx", (dY.dtype,), device, shape)
        elif p != 0:
            dx = torch.empty_like(dY)
        if dw is None:
            ws = None
        elif workspace is None:
            ws = _space(dY, _lib.load().dion_rms_norm_grad_workspace_size(rows, width))
        else:
            ws = _given_scratch(workspace, device)
        st = _lib.load().dion_rms_norm_grad(dY.data_ptr(), h.data_ptr(), w.data_ptr(), rstd.data_ptr(), _ptr(dsum),
                                            dh.data_ptr(), _ptr(dx), _ptr(dw), rows, width, float(p), _seed(seed, p, device),
                                            int(site), _DT[dY.dtype], _DT[h.dtype], _DT[w.dtype],
                                            _DT[w.dtype if dw is None else dw.dtype], int(bool(accumulate)), _ptr(ws),
                                            0 if ws is None else ws.numel(), handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_rms_norm_grad")
    return dh, dh if dx is None else dx


def gated_ffn_workspace_for(rows: int, width: int, hidden: int, device, dtype=torch.bfloat16, *, x_dtype=None,
                            for_grad: bool = False, saved: bool = True) -> torch.Tensor:
    """Scratch for one gated_ffn_ call, or with ``for_grad`` one gated_ffn_grad_ call (``saved``: given gate and up), of these
    sizes: fewer rows may need more."""
    x = _lib.E4M3 if x_dtype == E4M3 else _DT[dtype]
    return _scratch(int(_lib.load().dion_gated_ffn_workspace_size(rows, width, hidden, _DT[dtype], x,
                                                                  (1 if saved else 2) if for_grad else 0)), device)


def _block(X, Wg, Wu, Wd, act, scale):
    _need(Wg, "Wg", _DT)
    if Wg.dim() != 2:
        raise ValueError(f"Wg must be a matrix [hidden, width], got shape {tuple(Wg.shape)}")
    hidden, width = Wg.shape
    device, dtype = Wg.device, Wg.dtype
    _check(Wu, "Wu", (dtype,), device, Wg.shape)
    _check(Wd, "Wd", (dtype,), device, (width, hidden))
    _need(X, "X", (dtype,) if scale is None else _Q8, device)
    if X.dim() < 1 or X.shape[-1] != width:
        raise ValueError(f"X has shape {tuple(X.shape)}, expected [..., {width}]")
    if scale is not None:
        _check(scale, "scale", _F32, device, X.shape[:-1])
    if act not in _ACT:
        raise ValueError(f"act is {act!r}, expected one of {tuple(_ACT)}")
    return X.numel() // width, width, hidden, _DT[dtype], _DT[dtype] if scale is None else _lib.E4M3


def _kept(gate, up, dtype, device, shape) -> int:
    """Checks gate and up; what their form adds to the activation."""
    if (gate is None) != (up is None):
        raise ValueError("gate and up are kept together: give both or neither")
    if gate is None:
        return 0
    _check(gate, "gate", (dtype, torch.int16) if dtype == torch.bfloat16 else (dtype,), device, shape)
    _check(up, "up", (gate.dtype,), device, shape)
    return _lib.KEEP_EVEN if gate.dtype == torch.int16 else 0


def gated_ffn_(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, *, act: str = "silu",
               scale: torch.Tensor | None = None, gate: torch.Tensor | None = None, up: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gated feed-forward block ``(act(X Wg^T) * (X Wu^T)) Wd^T`` (dion_gated_ffn).

    X: [..., width]; Wg, Wu: [hidden, width]; Wd: [width, hidden]; all float32 or all bfloat16.  With ``scale`` (float32 per
    row) X is float8_e4m3fn and stands for ``X * scale``, as rms_norm_8bit_ leaves it.  act: "silu" or "gelu" (its tanh form).
    gate, up: [..., hidden], both or neither: filled with what gated_ffn_grad_ needs of the two projections, float32 for
    float32 weights and int16 for bfloat16 ones, whose bits are a form described in dion_block.h: at least as exact as
    bfloat16 from 2^-80 to 2^64 and three bits more so in [2^-8, 2^8).  (bfloat16 tensors are taken too.  Their bits are no
    bfloat16 numbers either, but a form that has one bit less than those outside [2^-8, 2^8).)
    Returns (or fills) out, [..., width] of the weights' type.
    """
    _no_graph("gated_ffn_", "gated_ffn_grad_", ("X", X), ("Wg", Wg), ("Wu", Wu), ("Wd", Wd), ("scale", scale), ("gate", gate), ("up", up),
              ("out", out))
    rows, width, hidden, dt, xt = _block(X, Wg, Wu, Wd, act, scale)
    device, dtype, inner = Wg.device, Wg.dtype, X.shape[:-1] + (hidden,)
    act = _ACT[act] | _kept(gate, up, dtype, device, inner)
    with _On(device, stream) as handle:
        if out is None:
            out = torch.empty_like(X, dtype=dtype)
        else:
            _check(out, "out", (dtype,), device, X.shape)
        ws = _space(Wg, _lib.load().dion_gated_ffn_workspace_size(rows, width, hidden, dt, xt, 0)) if workspace is None \
            else _given_scratch(workspace, device)
        st = _lib.load().dion_gated_ffn(X.data_ptr(), _ptr(scale), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), _ptr(gate),
                                        _ptr(up), out.data_ptr(), rows, width, hidden, act, xt, dt, ws.data_ptr(),
                                        ws.numel(), handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_gated_ffn")
    return out


def gated_ffn_grad_(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, dY: torch.Tensor,
                    gate: torch.Tensor | None = None, up: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                    dWg: torch.Tensor | None = None, dWu: torch.Tensor | None = None, dWd: torch.Tensor | None = None, *,
                    act: str = "silu", scale: torch.Tensor | None = None, accumulate: bool = False,
                    workspace: torch.Tensor | None = None, stream=None):
    """Gradients of gated_ffn_ (dion_gated_ffn_grad), into those of dX, dWg, dWu and dWd that are given; returns the four.

    dY: the output's gradient, [..., width] of the weights' type; gate, up: gated_ffn_'s for the same X, Wg, Wu, or both
    None, which forms them again.  dX: [..., width] of the weights' type; dWg and dWu (both or neither) and dWd: shaped as
    the weights, float32 or bfloat16, written, or added to with ``accumulate``.  What is not asked for costs no product.
    """
    rows, width, hidden, dt, xt = _block(X, Wg, Wu, Wd, act, scale)
    device, dtype, inner = Wg.device, Wg.dtype, X.shape[:-1] + (hidden,)
    _check(dY, "dY", (dtype,), device, X.shape)
    act = _ACT[act] | _kept(gate, up, dtype, device, inner)
    if dX is not None:
        _check(dX, "dX", (dtype,), device, X.shape)
    if (dWg is None) != (dWu is None):
        raise ValueError("dWg and dWu come from one product: give both or neither")
    dw = dtype
    for name, t, like in (("dWg", dWg, Wg), ("dWu", dWu, Wu), ("dWd", dWd, Wd)):
        if t is not None:
            _check(t, name, _DT, device, like.shape)
            dw = t.dtype
    if any(t is not None and t.dtype != dw for t in (dWg, dWu, dWd)):
        raise TypeError("dWg, dWu and dWd must have one dtype")
    with _On(device, stream) as handle:
        ws = _space(Wg, _lib.load().dion_gated_ffn_workspace_size(rows, width, hidden, dt, xt, 2 if gate is None else 1)) \
            if workspace is None else _given_scratch(workspace, device)
        st = _lib.load().dion_gated_ffn_grad(X.data_ptr(), _ptr(scale), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
                                             dY.data_ptr(), _ptr(gate), _ptr(up), _ptr(dX), _ptr(dWg), _ptr(dWu), _ptr(dWd),
                                             rows, width, hidden, act, xt, dt, _DT[dw], int(bool(accumulate)),
                                             ws.data_ptr(), ws.numel(), handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_gated_ffn_grad")
    return dX, dWg, dWu, dWd
