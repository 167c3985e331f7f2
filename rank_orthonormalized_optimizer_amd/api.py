"""torch-facing wrappers of dion_step_batched (marshalling only, no arithmetic)."""
from __future__ import annotations

import operator
from collections import OrderedDict
from functools import reduce

import torch

from . import _lib, block, vocab

_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


def _check(t: torch.Tensor, name: str, shape, dtypes) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a GPU, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def workspace_for(m: int, n: int, batch: int, rank: int, device) -> torch.Tensor:
    """Device scratch for one call (allocated by torch; 256-byte aligned)."""
    nbytes = _lib.workspace_size(m, n, batch, rank)
    ws = torch.empty(max(nbytes, 256) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + max(nbytes, 256)]


def step_(X: torch.Tensor, G: torch.Tensor, M: torch.Tensor, Q: torch.Tensor | None, rank: int,
          mu: float, lr: float, eps: float = 1e-8, *, workspace: torch.Tensor | None = None,
          flags: torch.Tensor | None = None, options: int = 0, stream=None, events=None,
          rmmc: torch.Tensor | None = None) -> None:
    """One Dion step on a stack, in place on X, M and Q.

    X, G: [b, m, n] float32 or bfloat16; M: [b, m, n] float32; Q: [b, n, rank] float32.
    ``flags`` (int32 [b], optional) receives the per-matrix FLAG_* bits.
    Enqueued on ``stream`` (default: torch's current stream) with no host sync.
    ``events``: optional NUM_PHASES + 1 recorded torch.cuda.Event objects, re-recorded at the
    phase boundaries of the step (profiling).
    ``rmmc`` (float32 [b], optional) receives each matrix's relative maximum momentum change
    max |M' - M| / max |M| over the step.
    """
    if X.dim() != 3:
        raise ValueError("X must be a stack [batch, m, n]; route 1-D parameters to AdamW or Lion")
    b, m, n = X.shape
    _check(X, "X", (b, m, n), tuple(_DT))
    _check(G, "G", (b, m, n), tuple(_DT))
    _check(M, "M", (b, m, n), (torch.float32,))
    if rank > 0:
        _check(Q, "Q", (b, n, rank), (torch.float32,))
    if flags is not None:
        _check(flags, "flags", (b,), (torch.int32,))
    if rmmc is not None:
        _check(rmmc, "rmmc", (b,), (torch.float32,))
    if workspace is None:
        workspace = workspace_for(m, n, b, rank, X.device)
    if stream is None:
        stream = torch.cuda.current_stream(X.device)
    st = _lib.step_batched_raw(X.data_ptr(), G.data_ptr(), M.data_ptr(), Q.data_ptr() if rank > 0 else 0,
                               m, n, b, rank, float(mu), float(lr), float(eps), _DT[X.dtype], _DT[G.dtype],
                               workspace.data_ptr(), workspace.numel(),
                               flags.data_ptr() if flags is not None else 0, int(options),
                               int(stream.cuda_stream),
                               None if events is None else [e.cuda_event for e in events],
                               rmmc.data_ptr() if rmmc is not None else 0)
    if st != _lib.OK:
        raise _lib.DionError(st)


class StickyF64Hint:
    """Host-side knowledge, gathered without a host sync, that a whole stack is on the fp64 chain.

    Under OPT_STICKY_F64 a matrix whose FLAG_F64 is set skips the fp32 attempt and keeps the
    flag, so once every flag is set the fp32 chain has no matrix left and OPT_FORCE_F64 gives
    the same kernels' work and bitwise the same results while not launching the (empty) fp32
    chain at all.  After each step the flags are copied to pinned host memory; the copy is
    looked at on a later step, once its event has completed.  Call ``reset()`` after changing
    the flags tensor by hand.
    """

    def __init__(self, flags: torch.Tensor):
        self.flags = flags
        self.host = torch.zeros(tuple(flags.shape), dtype=torch.int32, pin_memory=True)
        self.event = None
        self.all_f64 = False

    def reset(self) -> None:
        self.event = None
        self.all_f64 = False

    def options(self, base: int) -> int:
        if self.all_f64 and (base & _lib.OPT_STICKY_F64) and not (base & _lib.OPT_FORCE_F32):
            return base | _lib.OPT_FORCE_F64
        return base

    def after_step(self, stream) -> None:
        if self.all_f64:
            return
        if self.event is not None:
            if not self.event.query():
                return                       # the last copy is still in flight: look next step
            self.all_f64 = bool(((self.host & _lib.FLAG_F64) != 0).all())
            if self.all_f64:
                return
        with torch.cuda.stream(stream):
            self.host.copy_(self.flags, non_blocking=True)
            self.event = torch.cuda.Event()
            self.event.record(stream)


class DionStack:
    """Optimizer state (M, Q, flags, workspace) of one stack of same-shape matrices.

    ``rank_fraction`` picks r = floor(fraction * min(m, n)) (the rank-fraction
    knob of the rivista.ai Dion page) unless ``rank`` is given.  The fp64
    fallback is sticky by default: a matrix that needed it keeps it.
    """

    def __init__(self, batch: int, m: int, n: int, *, rank: int | None = None, rank_fraction: float = 0.25,
                 mu: float = 0.95, lr: float = 0.01, eps: float = 1e-8, device="cuda", sticky: bool = True,
                 seed: int = 0):
        self.batch, self.m, self.n = batch, m, n
        self.rank = int(rank if rank is not None else int(rank_fraction * min(m, n)))
        self.mu, self.lr, self.eps = mu, lr, eps
        self.options = _lib.OPT_STICKY_F64 if sticky else 0
        dev = torch.device(device)
        self.M = torch.zeros(batch, m, n, dtype=torch.float32, device=dev)
        gen = torch.Generator(device="cpu").manual_seed(seed)
        q = torch.randn(batch, n, self.rank, generator=gen, dtype=torch.float64)
        if self.rank:
            q /= q.norm(dim=1, keepdim=True)
        self.Q = q.to(torch.float32).to(dev).contiguous()
        self.flags = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.workspace = workspace_for(m, n, batch, self.rank, dev)
        self.hint = StickyF64Hint(self.flags) if sticky else None

    def step(self, X: torch.Tensor, G: torch.Tensor) -> None:
        opts = self.hint.options(self.options) if self.hint is not None else self.options
        stream = torch.cuda.current_stream(self.flags.device)
        step_(X, G, self.M, self.Q, self.rank, self.mu, self.lr, self.eps, workspace=self.workspace,
              flags=self.flags, options=opts, stream=stream)
        if self.hint is not None:
            self.hint.after_step(stream)

    def state_dict(self) -> dict:
        """The state a checkpoint needs, as CPU tensors: the momentum M, the right factor Q and
        the per-matrix flags (their fp64 mark keeps a matrix on the fp64 chain), with the
        sizes and hyper-parameters.  The workspace carries nothing from one step to the next, so
        a stack restored with load_state_dict continues bitwise as if it had not stopped."""
        return {"M": self.M.cpu(), "Q": self.Q.cpu(), "flags": self.flags.cpu(),
                "shape": [self.batch, self.m, self.n], "rank": self.rank, "mu": self.mu, "lr": self.lr,
                "eps": self.eps, "options": self.options}

    def load_state_dict(self, sd: dict) -> None:
        """Restore a state_dict() of a stack with the same sizes (copied into this stack's
        device tensors; the host's fp64 hint starts over, which selects the same work)."""
        if list(sd["shape"]) != [self.batch, self.m, self.n] or int(sd["rank"]) != self.rank:
            raise ValueError(f"state of a {sd['shape']} r={sd['rank']} stack, this one is "
                             f"{[self.batch, self.m, self.n]} r={self.rank}")
        self.M.copy_(sd["M"])
        self.Q.copy_(sd["Q"])
        self.flags.copy_(sd["flags"])
        self.mu, self.lr, self.eps, self.options = float(sd["mu"]), float(sd["lr"]), float(sd["eps"]), int(sd["options"])
        self.hint = StickyF64Hint(self.flags) if self.options & _lib.OPT_STICKY_F64 else None

    @property
    def P(self) -> torch.Tensor:
        """This step's orthonormal factor P [b, m, r] (fp32), read from the workspace."""
        n = self.batch * self.m * self.rank
        return self.workspace[:4 * n].view(torch.float32).view(self.batch, self.m, self.rank)


class GraphedStep:
    """One DionStack step captured in a HIP graph for fixed tensors, replayed by ``replay()``.

    The step's kernels and arguments are those of ``stack.step(X, G)`` at capture time
    (including the options the host hint has settled on), so a replay gives bitwise the result
    of an eager step on the same inputs, without the host launching each kernel.  ``G`` is read
    at replay time: refill it in place between replays.  Capture after at least one eager step
    (the sticky flags and the hint settle there); recapture if the options should change.
    """

    def __init__(self, stack: "DionStack", X: torch.Tensor, G: torch.Tensor):
        self.stack, self.X, self.G = stack, X, G
        dev = stack.flags.device
        opts = stack.hint.options(stack.options) if stack.hint is not None else stack.options
        cur = torch.cuda.current_stream(dev)
        cap = torch.cuda.Stream(device=dev)
        cap.wait_stream(cur)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(cap):
            self.graph.capture_begin()
            step_(X, G, stack.M, stack.Q, stack.rank, stack.mu, stack.lr, stack.eps, workspace=stack.workspace,
                  flags=stack.flags, options=opts, stream=cap)
            self.graph.capture_end()
        cur.wait_stream(cap)

    def replay(self) -> None:
        """Enqueue the captured step on torch's current stream."""
        self.graph.replay()


def group_matrices(params) -> "OrderedDict[tuple, list]":
    """Group 2-D tensors by (shape, dtype) into stackable lists; reject anything else.

    Dion updates 2-D weight matrices only; biases and other 1-D tensors go to
    AdamW or Lion, so they raise here instead of being silently skipped.
    """
    groups: "OrderedDict[tuple, list]" = OrderedDict()
    for i, p in enumerate(params):
        if p.dim() != 2:
            raise ValueError(f"parameter {i} has shape {tuple(p.shape)}: only 2-D matrices go to Dion")
        groups.setdefault((tuple(p.shape), p.dtype), []).append(p)
    return groups


def _flat_check(t: torch.Tensor, name: str, n: int, dtypes) -> None:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous GPU tensor")
    if t.numel() != n or t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.numel()} elements of {t.dtype}, expected {n} of {dtypes}")


def adamw_step_(param: torch.Tensor, grad: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, t: int,
                lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                *, stream=None) -> None:
    """One AdamW step (dion_adamw_step) on a contiguous tensor of any shape, in place; t counts from 1."""
    n = param.numel()
    _flat_check(param, "param", n, tuple(_DT))
    _flat_check(grad, "grad", n, tuple(_DT))
    _flat_check(exp_avg, "exp_avg", n, (torch.float32,))
    _flat_check(exp_avg_sq, "exp_avg_sq", n, (torch.float32,))
    if stream is None:
        stream = torch.cuda.current_stream(param.device)
    st = _lib.adamw_step_raw(param.data_ptr(), grad.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), n, int(t),
                             float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                             _DT[param.dtype], _DT[grad.dtype], int(stream.cuda_stream))
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_adamw_step")


def lambda_max_(W: torch.Tensor, k: int = 32, iters: int = 10, V0: torch.Tensor | None = None,
                out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """Multi-power-iteration estimate of lambda_max for each symmetric PSD matrix of the fp64
    stack W [b, r, r] (dion_lambda_max_batched; only the lower triangle is read).  V0 [b, r, k]
    fp64 or None for the library's start vectors.  Returns (or fills) fp64 [b] on W's device."""
    if not isinstance(W, torch.Tensor) or W.device.type != "cuda" or W.dtype != torch.float64 or W.dim() != 3 \
            or W.shape[1] != W.shape[2] or not W.is_contiguous():
        raise ValueError("W must be a contiguous fp64 GPU tensor [b, r, r]")
    b, r = int(W.shape[0]), int(W.shape[1])
    if V0 is not None:
        if V0.dtype != torch.float64 or tuple(V0.shape) != (b, r, k) or not V0.is_contiguous() or V0.device != W.device:
            raise ValueError(f"V0 must be a contiguous fp64 tensor [{b}, {r}, {k}] on W's device")
    if out is None:
        out = torch.empty(b, dtype=torch.float64, device=W.device)
    elif out.dtype != torch.float64 or out.numel() != b or not out.is_contiguous() or out.device != W.device:
        raise ValueError("out must be a contiguous fp64 tensor of b elements on W's device")
    nbytes = _lib.lambda_max_workspace_size(r, b, k)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=W.device)
    if stream is None:
        stream = torch.cuda.current_stream(W.device)
    st = _lib.lambda_max_raw(W.data_ptr(), r, b, 0 if V0 is None else V0.data_ptr(), int(k), int(iters),
                             out.data_ptr(), ws.data_ptr(), nbytes, int(stream.cuda_stream))
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_lambda_max_batched")
    return out


def lion_step_(param: torch.Tensor, grad: torch.Tensor, exp_avg: torch.Tensor, lr: float, beta1: float = 0.9,
               beta2: float = 0.99, weight_decay: float = 0.0, *, stream=None) -> None:
    """One Lion step (dion_lion_step) on a contiguous tensor of any shape, in place."""
    n = param.numel()
    _flat_check(param, "param", n, tuple(_DT))
    _flat_check(grad, "grad", n, tuple(_DT))
    _flat_check(exp_avg, "exp_avg", n, (torch.float32,))
    if stream is None:
        stream = torch.cuda.current_stream(param.device)
    st = _lib.lion_step_raw(param.data_ptr(), grad.data_ptr(), exp_avg.data_ptr(), n, float(lr), float(beta1),
                            float(beta2), float(weight_decay), _DT[param.dtype], _DT[grad.dtype],
                            int(stream.cuda_stream))
    if st != _lib.OK:
        raise _lib.DionError(st, "dion_lion_step")


class MixedDion:
    """Dion for the 2-D parameters, AdamW or Lion for the rest (rivista.ai, "Tecnicamente").

    ``params``: a list of GPU tensors.  2-D ones are grouped by (shape, dtype) into stacks
    (each step copies the group's weights and gradients into [b, m, n] stacks and back, since
    torch parameters are separate tensors); every other tensor gets element-wise state.
    ``step(grads)`` takes the gradients in the same order.

    The vocabulary matrices among the parameters (an embedding table, an output head, or one
    [vocab, width] matrix that is both) can be used through the optimizer, which then gathers their
    gradients itself: ``lookup`` and ``lookup_grad``, ``head_loss``; so can the parameters of the residual
    blocks between them: ``norm`` and ``norm_grad``, ``feed_forward`` and ``feed_forward_grad``.  All
    contributions since the last step add up (tied weights, microbatches), in float32 whatever the
    parameter's type, and ``step`` takes them where ``grads`` holds None.  Calls that gather, and ``step``, run on
    torch's current stream; a program that changes it between them orders the streams.
    """

    def __init__(self, params, *, lr: float = 0.01, mu: float = 0.95, rank_fraction: float = 0.25,
                 other: str = "adamw", other_lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.0):
        if other not in ("adamw", "lion"):
            raise ValueError("other must be 'adamw' or 'lion'")
        self.params = list(params)
        self.other, self.other_lr, self.betas, self.eps, self.wd = other, other_lr, betas, eps, weight_decay
        self.t = 0
        self.groups = []   # (indices, DionStack)
        mats = OrderedDict()
        for i, p in enumerate(self.params):
            if p.dim() == 2:
                mats.setdefault((tuple(p.shape), p.dtype), []).append(i)
        for (shape, _), idx in mats.items():
            st = DionStack(len(idx), shape[0], shape[1], rank_fraction=rank_fraction, mu=mu, lr=lr,
                           device=self.params[idx[0]].device)
            self.groups.append((idx, st))
        self.rest = [i for i, p in enumerate(self.params) if p.dim() != 2]
        self.state = {i: (torch.zeros(self.params[i].numel(), dtype=torch.float32, device=self.params[i].device),
                          torch.zeros(self.params[i].numel(), dtype=torch.float32, device=self.params[i].device)
                          if other == "adamw" else None) for i in self.rest}
        self.gathered = {}      # parameter index -> its gradient buffer, float32: bf16 would drop small contributions
        self.pending = set()    # those whose buffer holds contributions since the last step

    def _index(self, i: int) -> int:
        """i counted from the front, as the buffers are kept (-1 is the last parameter)."""
        n, k = len(self.params), operator.index(i)
        if not -n <= k < n:
            raise IndexError(f"parameter {k} of {n}")
        return k % n

    def _gather(self, i: int):
        """The gradient buffer of parameter i, and whether a contribution adds to what it holds."""
        if i not in self.gathered:
            self.gathered[i] = torch.empty(self.params[i].shape, dtype=torch.float32, device=self.params[i].device)
        return self.gathered[i], i in self.pending

    @torch.no_grad()
    def lookup(self, i: int, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
        """Rows ``scale * params[i][ids]`` (embedding_)."""
        return vocab.embedding_(ids, self.params[self._index(i)], scale)

    @torch.no_grad()
    def lookup_grad(self, i: int, ids: torch.Tensor, dY: torch.Tensor, scale: float = 1.0, *, padding_id: int = -1) -> None:
        """Add the table gradient of ``lookup(i, ids, scale)`` for the gradient ``dY`` of its rows (embedding_grad_)."""
        i = self._index(i)
        dW, add = self._gather(i)
        vocab.embedding_grad_(ids, dY, dW, scale, padding_id=padding_id, accumulate=add)
        self.pending.add(i)

    @torch.no_grad()
    def head_loss(self, i: int, H: torch.Tensor, targets: torch.Tensor, grad: torch.Tensor | None = None, *,
                  ignore_index: int = -100):
        """Cross entropy of the logits ``H params[i]^T`` (linear_cross_entropy_) and its gradients.

        ``grad``: float32, the loss's gradient per token or one element for all (default: the mean over
        the tokens that are not ignored).  Returns (per-token loss, dH) and adds the head's gradient.
        """
        i = self._index(i)
        W = self.params[i]
        loss, lse = vocab.linear_cross_entropy_(H, W, targets, ignore_index=ignore_index)
        if grad is None:
            grad = (targets != ignore_index).sum().clamp_(min=1).to(torch.float32).reciprocal_().reshape(1)
        dH = torch.empty_like(H)
        dW, add = self._gather(i)
        vocab.linear_cross_entropy_grad_(H, W, targets, lse, grad, dH, dW, ignore_index=ignore_index, accumulate=add)
        self.pending.add(i)
        return loss, dH

    @torch.no_grad()
    def norm(self, i: int, x: torch.Tensor, eps: float = 1e-6, *, eight: bool = False, **kw):
        """Root-mean-square norm with the weight ``params[i]`` (rms_norm_, or with ``eight`` rms_norm_8bit_; ``kw``: theirs)."""
        call = block.rms_norm_8bit_ if eight else block.rms_norm_
        return call(x, self.params[self._index(i)], eps, **kw)

    @torch.no_grad()
    def norm_grad(self, i: int, dY: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, *, dsum: torch.Tensor | None = None,
                  p: float = 0.0, seed: torch.Tensor | None = None, site: int = 0, dh: torch.Tensor | None = None,
                  dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
        """Gradients ``(dh, dx)`` of ``norm`` (rms_norm_grad_, with its arguments but for a stream: what is gathered belongs to
        the current one, as in every call that gathers); adds the weight's."""
        i = self._index(i)
        dw, add = self._gather(i)
        out = block.rms_norm_grad_(dY, h, self.params[i], rstd, dw, dsum=dsum, p=p, seed=seed, site=site, dh=dh, dx=dx,
                                   accumulate=add, workspace=workspace)
        self.pending.add(i)
        return out

    def _gated(self, weights):
        """The indexes of a feed-forward block's matrices (gate, up, down), three different ones."""
        idx = [self._index(i) for i in weights]
        if len(set(idx)) != 3:
            raise ValueError(f"a feed-forward block has three matrices (gate, up, down), got parameters {idx}")
        return idx

    @torch.no_grad()
    def feed_forward(self, weights, X: torch.Tensor, *, act: str = "silu", scale: torch.Tensor | None = None,
                     keep: bool = True):
        """Gated feed-forward block of the parameters ``weights`` = (gate, up, down) (gated_ffn_).

        Returns ``(Y, kept)``; ``kept`` goes to ``feed_forward_grad``, which without it (``keep`` False) forms the two
        projections again.
        """
        Wg, Wu, Wd = (self.params[i] for i in self._gated(weights))
        kept = None
        if keep:
            shape = X.shape[:-1] + Wg.shape[:1]
            form = torch.int16 if Wg.dtype == torch.bfloat16 else Wg.dtype   # (16 bits as exact as bfloat16 at any scale)
            kept = tuple(torch.empty(shape, dtype=form, device=Wg.device) for _ in range(2))
        return block.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale, gate=kept and kept[0], up=kept and kept[1]), kept

    @torch.no_grad()
    def feed_forward_grad(self, weights, X: torch.Tensor, dY: torch.Tensor, kept=None, *, act: str = "silu",
                          scale: torch.Tensor | None = None) -> torch.Tensor:
        """Gradient of ``X`` of the block ``feed_forward(weights, X)`` for the output's gradient ``dY`` (gated_ffn_grad_); adds
        the three matrices'."""
        idx = self._gated(weights)
        gathered = [self._gather(i) for i in idx]
        add = any(a for _, a in gathered)
        dX = torch.empty_like(dY)
        gate, up = kept or (None, None)
        if add:   # one of them has a gradient already: the others start from zero
            for dW, a in gathered:
                if not a:
                    dW.zero_()
        block.gated_ffn_grad_(X, *(self.params[i] for i in idx), dY, gate, up, dX, *(dW for dW, _ in gathered), act=act,
                              scale=scale, accumulate=add)
        self.pending.update(idx)
        return dX

    @torch.no_grad()
    def step(self, grads) -> None:
        grads = list(grads)
        if len(grads) < len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        for i, p in enumerate(self.params):   # everything is looked at before anything is updated
            if grads[i] is None and i not in self.pending:
                raise ValueError(f"no gradient for parameter {i}: none given and none gathered")
            if grads[i] is not None and i in self.pending:
                raise ValueError(f"parameter {i} has a gathered gradient; pass None for it")
            if grads[i] is None:
                grads[i] = self.gathered[i]
            if not isinstance(grads[i], torch.Tensor):
                raise TypeError(f"gradient of parameter {i} must be a torch.Tensor")
            if grads[i].numel() != p.numel() or (p.dim() == 2 and grads[i].shape != p.shape):
                raise ValueError(f"gradient of parameter {i} has shape {tuple(grads[i].shape)}, expected {tuple(p.shape)}")
            if grads[i].device != p.device:
                raise ValueError(f"gradient of parameter {i} lives on {grads[i].device}, expected {p.device}")
        for idx in [idx for idx, _ in self.groups] + [[i] for i in self.rest]:
            dtype = reduce(torch.promote_types, [grads[i].dtype for i in idx])   # of a stack's gradients together
            if dtype not in _DT:
                raise TypeError(f"gradients of parameters {idx} have dtype {dtype}, expected one of {tuple(_DT)}")
        self.t += 1
        for idx, st in self.groups:
            X = torch.stack([self.params[i] for i in idx]).contiguous()
            G = torch.stack([grads[i] for i in idx]).contiguous()   # bf16 beside a gathered float32: float32
            st.step(X, G)
            for k, i in enumerate(idx):
                self.params[i].copy_(X[k])
        for i in self.rest:
            p, g = self.params[i], grads[i].contiguous()
            m, v = self.state[i]
            if self.other == "adamw":
                adamw_step_(p, g, m, v, self.t, self.other_lr, self.betas[0], self.betas[1], self.eps, self.wd)
            else:
                lion_step_(p, g, m, self.other_lr, self.betas[0], self.betas[1], self.wd)
        self.pending.clear()   # only now: a refused step leaves them for the next
