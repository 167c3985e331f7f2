"""The residual blocks' C ABI and Python wrappers on the host (no GPU needed): every declared symbol is
exported, sizes are consistent, and invalid calls are refused before any HIP call."""
import os
import re

import pytest
import torch

import rank_orthonormalized_optimizer_amd as dion
from rank_orthonormalized_optimizer_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dion_block.h")
BASE, GB = 1 << 40, 1 << 30   # fake device addresses, never dereferenced


def P(gib, off=0):
    return BASE + gib * GB + off


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dion_(?!activation)\w+)\s*\(", text)))
    assert set(names) == set(_lib.BLOCK_EXPORTS)
    lib = dion.load()
    for name in names:
        assert hasattr(lib, name), name
    assert re.search(r"#define DION_E4M3 2", text) and _lib.E4M3 == 2
    assert re.search(r"DION_SILU = 0, DION_GELU = 1", text) and (_lib.SILU, _lib.GELU) == (0, 1)
    assert re.search(r"DION_BLOCK_MAX_ROWS \(\(int64_t\)1 << 20\)", text) and _lib.BLOCK_MAX_ROWS == 1 << 20


def dropout(**kw):
    a = dict(x=P(0), residual=P(1), out=P(2), n=100, p=0.1, seed=P(3), site=0, xt=1, ot=1, stream=0)
    a.update(kw)
    return int(_lib.load().dion_dropout(*a.values()))


def norm(**kw):
    a = dict(x=P(0), residual=P(1), w=P(2), h=P(3), y=P(4), scale=0, rstd=P(6), rows=10, width=24, eps=1e-6, p=0.1, seed=P(7),
             site=0, xt=1, st=1, wt=1, yt=1, stream=0)
    a.update(kw)
    return int(_lib.load().dion_rms_norm(*a.values()))


def grad(**kw):
    a = dict(dY=P(0), h=P(1), w=P(2), rstd=P(3), dsum=P(4), dh=P(5), dx=P(6), dw=P(7), rows=10, width=24, p=0.1, seed=P(8), site=0,
             yt=1, st=1, wt=1, dwt=1, acc=0, ws=P(9), nbytes=GB, stream=0)
    a.update(kw)
    return int(_lib.load().dion_rms_norm_grad(*a.values()))


def ffn(**kw):
    a = dict(X=P(0), scale=0, Wg=P(1), Wu=P(2), Wd=P(3), gate=P(4), up=P(5), Y=P(6), rows=100, width=24, hidden=40, act=0, xt=1, dt=1,
             ws=P(7), nbytes=GB, stream=0)
    a.update(kw)
    return int(_lib.load().dion_gated_ffn(*a.values()))


def ffn_grad(**kw):
    a = dict(X=P(0), scale=0, Wg=P(1), Wu=P(2), Wd=P(3), dY=P(4), gate=P(5), up=P(6), dX=P(7), dWg=P(8), dWu=P(9), dWd=P(10), rows=10,
             width=24, hidden=40, act=0, xt=1, dt=1, dwt=1, acc=0, ws=P(11), nbytes=GB, stream=0)
    a.update(kw)
    return int(_lib.load().dion_gated_ffn_grad(*a.values()))


SIZES = [(dict(rows=-1), _lib.ERR_SHAPE), (dict(rows=(1 << 20) + 1), _lib.ERR_SHAPE), (dict(width=0), _lib.ERR_SHAPE),
         (dict(width=(1 << 16) + 1), _lib.ERR_SHAPE)]


@pytest.mark.parametrize("call", [norm, grad, ffn, ffn_grad])
@pytest.mark.parametrize("kw,status", SIZES)
def test_sizes_refused(call, kw, status):
    assert call(**kw) == status


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("call,kw,status", [
    (dropout, dict(n=-1), _lib.ERR_SHAPE), (dropout, dict(n=(1 << 36) + 1), _lib.ERR_SHAPE), (dropout, dict(p=1.0), _lib.ERR_HYPER),
    (dropout, dict(p=-0.1), _lib.ERR_HYPER), (dropout, dict(p=NAN), _lib.ERR_HYPER), (dropout, dict(xt=2), _lib.ERR_DTYPE),
    (dropout, dict(ot=-1), _lib.ERR_DTYPE), (dropout, dict(x=0), _lib.ERR_NULL), (dropout, dict(out=0), _lib.ERR_NULL),
    (dropout, dict(seed=0), _lib.ERR_NULL), (dropout, dict(x=P(0, 8)), _lib.ERR_ALIGN), (dropout, dict(seed=P(3, 4)), _lib.ERR_ALIGN),
    (dropout, dict(residual=P(1, 2)), _lib.ERR_ALIGN), (dropout, dict(out=P(0, 16)), _lib.ERR_OVERLAP),
    (dropout, dict(out=P(1, 16)), _lib.ERR_OVERLAP), (dropout, dict(seed=P(2, 8)), _lib.ERR_OVERLAP),
    (norm, dict(eps=-1e-9), _lib.ERR_HYPER), (norm, dict(eps=INF), _lib.ERR_HYPER), (norm, dict(eps=NAN), _lib.ERR_HYPER),
    (norm, dict(p=1.5), _lib.ERR_HYPER), (norm, dict(xt=2), _lib.ERR_DTYPE), (norm, dict(st=2), _lib.ERR_DTYPE),
    (norm, dict(wt=3), _lib.ERR_DTYPE), (norm, dict(yt=3), _lib.ERR_DTYPE), (norm, dict(x=0), _lib.ERR_NULL),
    (norm, dict(w=0), _lib.ERR_NULL), (norm, dict(y=0), _lib.ERR_NULL), (norm, dict(seed=0), _lib.ERR_NULL),
    (norm, dict(yt=2), _lib.ERR_NULL), (norm, dict(scale=P(5)), _lib.ERR_NULL), (norm, dict(w=P(2, 4)), _lib.ERR_ALIGN),
    (norm, dict(rstd=P(6, 2)), _lib.ERR_ALIGN), (norm, dict(yt=2, scale=P(5, 1)), _lib.ERR_ALIGN),
    (norm, dict(h=P(0)), _lib.ERR_OVERLAP), (norm, dict(h=P(1, 16)), _lib.ERR_OVERLAP), (norm, dict(y=P(1)), _lib.ERR_OVERLAP),
    (norm, dict(rstd=P(4, 16)), _lib.ERR_OVERLAP),
    (grad, dict(p=1.0), _lib.ERR_HYPER), (grad, dict(yt=2), _lib.ERR_DTYPE), (grad, dict(st=2), _lib.ERR_DTYPE),
    (grad, dict(wt=2), _lib.ERR_DTYPE), (grad, dict(dwt=2), _lib.ERR_DTYPE), (grad, dict(acc=2), _lib.ERR_OPTION),
    (grad, dict(dY=0), _lib.ERR_NULL), (grad, dict(h=0), _lib.ERR_NULL), (grad, dict(w=0), _lib.ERR_NULL),
    (grad, dict(rstd=0), _lib.ERR_NULL), (grad, dict(dh=0), _lib.ERR_NULL), (grad, dict(seed=0), _lib.ERR_NULL),
    (grad, dict(ws=0), _lib.ERR_NULL), (grad, dict(dx=P(6, 4)), _lib.ERR_ALIGN), (grad, dict(ws=P(9, 64)), _lib.ERR_ALIGN),
    (grad, dict(nbytes=16), _lib.ERR_WORKSPACE), (grad, dict(dh=P(1)), _lib.ERR_OVERLAP), (grad, dict(dx=P(5, 16)), _lib.ERR_OVERLAP),
    (grad, dict(dh=P(4, 16)), _lib.ERR_OVERLAP), (grad, dict(dx=P(4)), _lib.ERR_OVERLAP), (grad, dict(dw=P(2)), _lib.ERR_OVERLAP),
    (ffn, dict(hidden=0), _lib.ERR_SHAPE), (ffn, dict(hidden=(1 << 17) + 1), _lib.ERR_SHAPE), (ffn, dict(act=2), _lib.ERR_OPTION),
    (ffn, dict(dt=2), _lib.ERR_DTYPE), (ffn, dict(xt=0), _lib.ERR_DTYPE), (ffn, dict(X=0), _lib.ERR_NULL), (ffn, dict(Wg=0), _lib.ERR_NULL),
    (ffn, dict(Wu=0), _lib.ERR_NULL), (ffn, dict(Wd=0), _lib.ERR_NULL), (ffn, dict(Y=0), _lib.ERR_NULL), (ffn, dict(ws=0), _lib.ERR_NULL),
    (ffn, dict(gate=0), _lib.ERR_NULL), (ffn, dict(up=0), _lib.ERR_NULL), (ffn, dict(scale=P(8)), _lib.ERR_NULL),
    (ffn, dict(xt=2), _lib.ERR_NULL), (ffn, dict(Wg=P(1, 8)), _lib.ERR_ALIGN), (ffn, dict(ws=P(7, 16)), _lib.ERR_ALIGN),
    (ffn, dict(xt=2, scale=P(8, 2)), _lib.ERR_ALIGN), (ffn, dict(nbytes=100), _lib.ERR_WORKSPACE), (ffn, dict(Y=P(0)), _lib.ERR_OVERLAP),
    (ffn, dict(up=P(4, 32)), _lib.ERR_OVERLAP), (ffn, dict(Y=P(7, 256)), _lib.ERR_OVERLAP), (ffn, dict(gate=P(3)), _lib.ERR_OVERLAP),
    (ffn_grad, dict(hidden=0), _lib.ERR_SHAPE), (ffn_grad, dict(act=-1), _lib.ERR_OPTION), (ffn_grad, dict(acc=2), _lib.ERR_OPTION),
    (ffn_grad, dict(dwt=2), _lib.ERR_DTYPE), (ffn_grad, dict(dX=0, dWg=0, dWu=0, dWd=0), _lib.ERR_NULL),
    (ffn_grad, dict(dWg=0), _lib.ERR_NULL), (ffn_grad, dict(gate=0), _lib.ERR_NULL), (ffn_grad, dict(dY=0), _lib.ERR_NULL),
    (ffn_grad, dict(ws=0), _lib.ERR_NULL), (ffn_grad, dict(dWd=P(10, 8)), _lib.ERR_ALIGN), (ffn_grad, dict(nbytes=1), _lib.ERR_WORKSPACE),
    (ffn_grad, dict(dX=P(4)), _lib.ERR_OVERLAP), (ffn_grad, dict(dWu=P(8)), _lib.ERR_OVERLAP), (ffn_grad, dict(dX=P(5)), _lib.ERR_OVERLAP),
])
def test_calls_refused(call, kw, status):
    assert call(**kw) == status


def test_empty_calls_do_nothing():
    assert dropout(n=0, x=0, residual=0, out=0, seed=0) == _lib.OK
    assert norm(rows=0, x=0, w=0, y=0, seed=0) == _lib.OK
    assert grad(rows=0, dw=0, dY=0, h=0, w=0, rstd=0, dh=0, ws=0) == _lib.OK
    assert grad(rows=0, acc=1, dY=0, h=0, w=0, rstd=0, dh=0, ws=0) == _lib.OK
    assert ffn(rows=0, X=0, Y=0, ws=0) == _lib.OK
    assert ffn_grad(rows=0, acc=1, X=0, dY=0, ws=0) == _lib.OK and ffn_grad(rows=0, dWg=0, dWu=0, dWd=0, X=0, dY=0, ws=0) == _lib.OK


def test_workspace_sizes():
    lib = dion.load()
    g = lib.dion_rms_norm_grad_workspace_size
    assert g(-1, 8) == 0 and g(8, 0) == 0 and g(0, 8) == 0 and g(1, 4096) == 0 and 0 < g(1000, 64) <= g(100000, 64)
    f = lib.dion_gated_ffn_workspace_size
    assert f(-1, 8, 8, 1, 1, 0) == 0 and f(8, 8, 0, 1, 1, 0) == 0 and f(8, 8, 8, 2, 2, 0) == 0 and f(8, 8, 8, 1, 0, 0) == 0
    assert f(8, 8, 8, 1, 1, 3) == 0
    assert 0 < f(512, 256, 512, 1, 1, 0) < f(512, 256, 512, 1, 1, 1) < f(512, 256, 512, 1, 1, 2)
    assert f(512, 256, 512, 1, 1, 0) < f(512, 256, 512, 1, 2, 0) and f(512, 256, 512, 0, 2, 1) > 0


def test_wrappers_refuse_cpu_tensors_and_wrong_arguments():
    x, w, W = torch.zeros(3, 8), torch.zeros(8), torch.zeros(16, 8)
    for call in (lambda: dion.dropout_(x, 0.1), lambda: dion.rms_norm_(x, w), lambda: dion.rms_norm_8bit_(x, w),
                 lambda: dion.rms_norm_grad_(x, x, w, torch.zeros(3)), lambda: dion.gated_ffn_(x, W, W, W.t().contiguous()),
                 lambda: dion.gated_ffn_grad_(x, W, W, W.t().contiguous(), x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        dion.rms_norm_([1.0], w)


@pytest.mark.parametrize("call", ["dropout_", "rms_norm_", "rms_norm_8bit_", "gated_ffn_"])
def test_tensors_that_require_a_gradient_refused(call):
    x, w, W = torch.zeros(3, 8, requires_grad=True), torch.zeros(8), torch.zeros(16, 8)
    args = {"dropout_": (x, 0.1), "rms_norm_": (x, w), "rms_norm_8bit_": (x, w), "gated_ffn_": (x, W, W, W.t().contiguous())}[call]
    with pytest.raises(ValueError, match="requires a gradient"):
        getattr(dion, call)(*args)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):   # taken, up to the next check
        getattr(dion, call)(*args)
