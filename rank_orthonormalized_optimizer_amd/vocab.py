"""torch-facing wrappers of include/dion_vocab.h: the operators over a language model's vocabulary
matrices (marshalling only, no arithmetic).

Tensors are contiguous and on one GPU; everything is enqueued on ``stream`` (default: torch's
current stream of that GPU) with no host sync.  Scratch and outputs that are not given are
allocated by torch on that stream.

No call records a graph for autograd: gradients are calls of their own (``embedding_grad_``,
``linear_cross_entropy_grad_``).  Where autograd would expect one, ``embedding_`` and
``linear_cross_entropy_`` refuse tensors that require a gradient: call them under
``torch.no_grad()`` or on detached tensors.
"""
from __future__ import annotations

import torch

from . import _lib

_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}
_IT = {torch.int32: _lib.I32, torch.int64: _lib.I64}


def _need(t, name: str, dtypes, device=None, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a GPU, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} lives on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _no_graph(call: str, **tensors) -> None:
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{call} records no graph, but {name} requires a gradient: call it under torch.no_grad() "
                                 f"or detach {name}, and {call[:-1]}_grad_ for the gradient")


def _matrix(t, name: str, device=None):
    _need(t, name, _DT, device)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix [vocab, width], got shape {tuple(t.shape)}")
    return t.shape


class _On:
    """The stream a call runs on.  Inside the block torch's current device is the tensors', and its current
    stream the one given, so that scratch allocated there is reused in that stream's order."""
    __slots__ = ("handle", "guard")

    def __init__(self, device, stream):
        if stream is None:   # the raw handle: a stream object costs as much as a third of a small call
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
            self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        else:
            if stream.device != device:
                raise ValueError(f"stream of {stream.device} for tensors on {device}")
            self.handle = stream.cuda_stream
            self.guard = torch.cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _scratch(nbytes: int, device) -> torch.Tensor:
    """Device scratch (torch's allocations are 512-byte aligned)."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _given_scratch(ws, device) -> torch.Tensor:
    _need(ws, "workspace", (torch.uint8,), device)
    return ws


def embedding_(ids: torch.Tensor, W: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None, *,
               stream=None) -> torch.Tensor:
    """Embedding lookup ``out[t] = scale * W[ids[t]]`` (dion_embedding), rounded once to ``out``'s type.

    ids: int32 or int64 of any shape; W: [vocab, width] float32 or bfloat16; out: ids' shape + [width],
    float32 or bfloat16 (default: W's type).  An id outside [0, vocab) gives a row of NaN.
    """
    _no_graph("embedding_", W=W, out=out)
    vocab, width = _matrix(W, "W")
    device = W.device
    _need(ids, "ids", _IT, device)
    with _On(device, stream) as handle:
        shape = ids.shape + (width,)
        if out is None:
            out = torch.empty(shape, dtype=W.dtype, device=device)
        else:
            _need(out, "out", _DT, device, shape)
        st = _lib.load().dion_embedding(ids.data_ptr(), W.data_ptr(), out.data_ptr(), ids.numel(), vocab, width,
                                        float(scale), _IT[ids.dtype], _DT[W.dtype], _DT[out.dtype], handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_embedding")
    return out


def embedding_grad_workspace_for(tokens: int, vocab: int, width: int, device) -> torch.Tensor:
    """Scratch for one embedding_grad_ call of these sizes."""
    return _scratch(int(_lib.load().dion_embedding_grad_workspace_size(tokens, vocab, width)), device)


def embedding_grad_(ids: torch.Tensor, dY: torch.Tensor, dW: torch.Tensor, scale: float = 1.0, *,
                    padding_id: int = -1, accumulate: bool = False, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Gradient of the lookup's table, ``dW[v] (+)= scale * sum of dY[t] over ids[t] = v`` (dion_embedding_grad).

    ids: int32 or int64; dY: ids' shape + [width]; dW: [vocab, width], written whole, or added to with
    ``accumulate`` (the head's gradient of tied weights, earlier microbatches).  dY and dW are float32 or
    bfloat16, independently.  Ids equal to ``padding_id`` or outside [0, vocab) leave no gradient.
    """
    vocab, width = _matrix(dW, "dW")
    device = dW.device
    _need(ids, "ids", _IT, device)
    _need(dY, "dY", _DT, device, ids.shape + (width,))
    tokens = ids.numel()
    with _On(device, stream) as handle:
        ws = embedding_grad_workspace_for(tokens, vocab, width, device) if workspace is None \
            else _given_scratch(workspace, device)
        st = _lib.load().dion_embedding_grad(ids.data_ptr(), dY.data_ptr(), dW.data_ptr(), tokens, vocab, width,
                                             float(scale), int(padding_id), _IT[ids.dtype], _DT[dY.dtype],
                                             _DT[dW.dtype], int(bool(accumulate)), ws.data_ptr(), ws.numel(), handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_embedding_grad")
    return dW


def linear_cross_entropy_workspace_for(tokens: int, vocab: int, width: int, device, dtype=torch.bfloat16, *,
                                       dw_dtype=None, for_grad: bool = False) -> torch.Tensor:
    """Scratch for one linear_cross_entropy_ call, or with ``for_grad`` one linear_cross_entropy_grad_ call."""
    return _scratch(int(_lib.load().dion_linear_xent_workspace_size(tokens, vocab, width, _DT[dtype],
                                                                    _DT[dw_dtype or dtype], int(for_grad))), device)


def _head(H, W, targets):
    vocab, width = _matrix(W, "W")
    _need(targets, "targets", _IT, W.device)
    _need(H, "H", (W.dtype,), W.device, targets.shape + (width,))
    return targets.numel(), vocab, width


def linear_cross_entropy_(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                          loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None):
    """Softmax cross entropy of the logits ``H W^T`` per token, which are not kept (dion_linear_xent).

    H: targets' shape + [width]; W: [vocab, width] of the same type, float32 or bfloat16; targets: int32 or
    int64.  Returns (or fills) float32 ``loss`` and ``lse`` (log-sum-exp of the logits) of targets' shape: 0
    where the target is ``ignore_index``; NaN loss for any other target outside [0, vocab).
    """
    _no_graph("linear_cross_entropy_", H=H, W=W, loss=loss, lse=lse)
    tokens, vocab, width = _head(H, W, targets)
    device = W.device
    with _On(device, stream) as handle:
        if loss is None:
            loss = torch.empty(targets.shape, dtype=torch.float32, device=device)
        else:
            _need(loss, "loss", (torch.float32,), device, targets.shape)
        if lse is None:
            lse = torch.empty(targets.shape, dtype=torch.float32, device=device)
        else:
            _need(lse, "lse", (torch.float32,), device, targets.shape)
        ws = linear_cross_entropy_workspace_for(tokens, vocab, width, device, W.dtype) if workspace is None \
            else _given_scratch(workspace, device)
        st = _lib.load().dion_linear_xent(H.data_ptr(), W.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                                          tokens, vocab, width, int(ignore_index), _IT[targets.dtype], _DT[W.dtype],
                                          ws.data_ptr(), ws.numel(), handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_linear_xent")
    return loss, lse


def linear_cross_entropy_grad_(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                               grad: torch.Tensor, dH: torch.Tensor | None = None, dW: torch.Tensor | None = None, *,
                               ignore_index: int = -100, accumulate: bool = False,
                               workspace: torch.Tensor | None = None, stream=None):
    """Gradients of ``sum(grad * loss)`` (dion_linear_xent_grad), into ``dH`` and ``dW``; returns both.

    lse: linear_cross_entropy_'s for the same H, W, targets; grad: float32, of targets' shape or one element for
    every token (1 / count for a mean).  dH (H's shape and type) and dW ([vocab, width], float32 or bfloat16) are
    written; one of them may be None, which saves its product.  An fp32 dW of bf16 operands is fp32-accurate and takes
    three times the product of a bf16 one, and its workspace.  ``accumulate`` adds to dW instead.  Ignored tokens
    get zeros in dH and leave nothing in dW.
    """
    tokens, vocab, width = _head(H, W, targets)
    device = W.device
    _need(lse, "lse", (torch.float32,), device, targets.shape)
    _need(grad, "grad", (torch.float32,), device)
    if grad.numel() != 1 and grad.shape != targets.shape:
        raise ValueError(f"grad has shape {tuple(grad.shape)}, expected {tuple(targets.shape)} or one element")
    if dH is not None:
        _need(dH, "dH", (H.dtype,), device, H.shape)
    if dW is not None:
        _need(dW, "dW", _DT, device, W.shape)
    dw = W.dtype if dW is None else dW.dtype
    with _On(device, stream) as handle:
        ws = linear_cross_entropy_workspace_for(tokens, vocab, width, device, W.dtype, dw_dtype=dw, for_grad=True) \
            if workspace is None else _given_scratch(workspace, device)
        st = _lib.load().dion_linear_xent_grad(H.data_ptr(), W.data_ptr(), targets.data_ptr(), lse.data_ptr(),
                                               grad.data_ptr(), grad.numel(), None if dH is None else dH.data_ptr(),
                                               None if dW is None else dW.data_ptr(), tokens, vocab, width,
                                               int(ignore_index), _IT[targets.dtype], _DT[W.dtype], _DT[dw],
                                               int(bool(accumulate)), ws.data_ptr(), ws.numel(), handle)
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_linear_xent_grad")
    return dH, dW
