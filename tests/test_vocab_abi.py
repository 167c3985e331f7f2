"""The vocabulary operators' C ABI and Python wrappers on the host (no GPU needed): every declared
symbol is exported, sizes are consistent, and invalid calls are refused before any HIP call."""
import os
import re

import pytest
import torch

import rank_orthonormalized_optimizer_amd as dion
from rank_orthonormalized_optimizer_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dion_vocab.h")
BASE, GB = 1 << 40, 1 << 30   # fake device addresses, never dereferenced


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dion_\w+)\s*\(", text)))
    assert set(names) == set(_lib.VOCAB_EXPORTS)
    lib = dion.load()
    for name in names:
        assert hasattr(lib, name), name
    assert re.search(r"DION_I32 = 0, DION_I64 = 1", text) and (_lib.I32, _lib.I64) == (0, 1)
    assert re.search(r"DION_VOCAB_MAX_TOKENS \(\(int64_t\)1 << 20\)", text) and _lib.VOCAB_MAX_TOKENS == 1 << 20


def lookup(**kw):
    a = dict(ids=BASE, W=BASE + GB, out=BASE + 2 * GB, tokens=10, vocab=100, width=24, scale=1.0, it=0, wt=1, ot=1, stream=0)
    a.update(kw)
    return int(_lib.load().dion_embedding(*a.values()))


def table(**kw):
    a = dict(ids=BASE, dY=BASE + GB, dW=BASE + 2 * GB, tokens=10, vocab=100, width=24, scale=1.0, pad=-1, it=1, yt=1, wt=0,
             acc=0, ws=BASE + 3 * GB, nbytes=GB, stream=0)
    a.update(kw)
    return int(_lib.load().dion_embedding_grad(*a.values()))


def loss(**kw):
    a = dict(H=BASE, W=BASE + GB, y=BASE + 2 * GB, loss=BASE + 3 * GB, lse=BASE + 4 * GB, tokens=10, vocab=100, width=24,
             ignore=-100, yt=1, dt=1, ws=BASE + 5 * GB, nbytes=4 * GB, stream=0)
    a.update(kw)
    return int(_lib.load().dion_linear_xent(*a.values()))


def grad(**kw):
    a = dict(H=BASE, W=BASE + GB, y=BASE + 2 * GB, lse=BASE + 3 * GB, g=BASE + 4 * GB, gn=1, dH=BASE + 5 * GB,
             dW=BASE + 6 * GB, tokens=10, vocab=100, width=24, ignore=-100, yt=1, dt=1, dwt=1, acc=0, ws=BASE + 8 * GB,
             nbytes=4 * GB, stream=0)
    a.update(kw)
    return int(_lib.load().dion_linear_xent_grad(*a.values()))


SIZES = [(dict(tokens=-1), _lib.ERR_SHAPE), (dict(tokens=(1 << 20) + 1), _lib.ERR_SHAPE), (dict(vocab=0), _lib.ERR_SHAPE),
         (dict(vocab=1 << 24), _lib.ERR_SHAPE), (dict(width=0), _lib.ERR_SHAPE), (dict(width=(1 << 16) + 1), _lib.ERR_SHAPE)]


@pytest.mark.parametrize("call", [lookup, table, loss, grad])
@pytest.mark.parametrize("kw,status", SIZES)
def test_sizes_refused(call, kw, status):
    if call is grad and "tokens" in kw:
        kw = dict(kw, gn=1)
    assert call(**kw) == status


@pytest.mark.parametrize("call,kw,status", [
    (lookup, dict(scale=float("inf")), _lib.ERR_HYPER), (lookup, dict(scale=float("nan")), _lib.ERR_HYPER),
    (lookup, dict(it=2), _lib.ERR_DTYPE), (lookup, dict(wt=2), _lib.ERR_DTYPE), (lookup, dict(ot=-1), _lib.ERR_DTYPE),
    (lookup, dict(ids=0), _lib.ERR_NULL), (lookup, dict(W=0), _lib.ERR_NULL), (lookup, dict(out=0), _lib.ERR_NULL),
    (lookup, dict(ids=BASE + 2), _lib.ERR_ALIGN), (lookup, dict(it=1, ids=BASE + 4), _lib.ERR_ALIGN),
    (lookup, dict(W=BASE + GB + 8), _lib.ERR_ALIGN), (lookup, dict(out=BASE + 2 * GB + 2), _lib.ERR_ALIGN),
    (lookup, dict(out=BASE + GB + 4784), _lib.ERR_OVERLAP), (lookup, dict(out=BASE + 32), _lib.ERR_OVERLAP),
    (table, dict(scale=float("nan")), _lib.ERR_HYPER), (table, dict(it=-1), _lib.ERR_DTYPE), (table, dict(yt=7), _lib.ERR_DTYPE),
    (table, dict(wt=2), _lib.ERR_DTYPE), (table, dict(acc=2), _lib.ERR_OPTION), (table, dict(ids=0), _lib.ERR_NULL),
    (table, dict(dY=0), _lib.ERR_NULL), (table, dict(dW=0), _lib.ERR_NULL), (table, dict(ws=0), _lib.ERR_NULL),
    (table, dict(ids=BASE + 4), _lib.ERR_ALIGN), (table, dict(dW=BASE + 2 * GB + 4), _lib.ERR_ALIGN),
    (table, dict(ws=BASE + 3 * GB + 16), _lib.ERR_ALIGN), (table, dict(nbytes=255), _lib.ERR_WORKSPACE),
    (table, dict(dY=BASE + 2 * GB + 16), _lib.ERR_OVERLAP),
    (loss, dict(yt=3), _lib.ERR_DTYPE), (loss, dict(dt=2), _lib.ERR_DTYPE), (loss, dict(H=0), _lib.ERR_NULL),
    (loss, dict(y=0), _lib.ERR_NULL), (loss, dict(loss=0), _lib.ERR_NULL), (loss, dict(lse=0), _lib.ERR_NULL),
    (loss, dict(ws=0), _lib.ERR_NULL), (loss, dict(W=BASE + GB + 4), _lib.ERR_ALIGN), (loss, dict(loss=BASE + 3 * GB + 2), _lib.ERR_ALIGN),
    (loss, dict(y=BASE + 2 * GB + 4), _lib.ERR_ALIGN), (loss, dict(nbytes=1000), _lib.ERR_WORKSPACE),
    (loss, dict(lse=BASE + 3 * GB + 36), _lib.ERR_OVERLAP), (loss, dict(loss=BASE + 16), _lib.ERR_OVERLAP),
    (grad, dict(gn=2), _lib.ERR_SHAPE), (grad, dict(gn=0), _lib.ERR_SHAPE), (grad, dict(dwt=2), _lib.ERR_DTYPE),
    (grad, dict(acc=-1), _lib.ERR_OPTION), (grad, dict(dH=0, dW=0), _lib.ERR_NULL), (grad, dict(lse=0), _lib.ERR_NULL),
    (grad, dict(g=0), _lib.ERR_NULL), (grad, dict(g=BASE + 4 * GB + 2), _lib.ERR_ALIGN), (grad, dict(dH=BASE + 5 * GB + 8), _lib.ERR_ALIGN),
    (grad, dict(ws=BASE + 8 * GB + 128), _lib.ERR_ALIGN), (grad, dict(nbytes=0), _lib.ERR_WORKSPACE),
    (grad, dict(dH=BASE), _lib.ERR_OVERLAP), (grad, dict(dW=BASE + GB), _lib.ERR_OVERLAP),
    (grad, dict(dW=BASE + 5 * GB + 16), _lib.ERR_OVERLAP),
])
def test_calls_refused(call, kw, status):
    assert call(**kw) == status


def test_overlapping_table_workspace_refused():
    assert table(ws=BASE + 2 * GB + 256) == _lib.ERR_OVERLAP     # inside dW
    assert table(ids=BASE + 3 * GB) == _lib.ERR_OVERLAP          # ids inside the workspace


def test_empty_calls_do_nothing():
    assert lookup(tokens=0, ids=0, W=0, out=0) == _lib.OK
    assert table(tokens=0, acc=1, ids=0, dY=0, dW=0, ws=0, nbytes=0) == _lib.OK
    assert loss(tokens=0, H=0, W=0, y=0, loss=0, lse=0, ws=0, nbytes=0) == _lib.OK
    assert grad(tokens=0, gn=0, acc=1, H=0, W=0, y=0, lse=0, g=0, ws=0) == _lib.OK
    assert grad(tokens=0, gn=1, dW=0, H=0, W=0, y=0, lse=0, g=0, ws=0) == _lib.OK


def test_workspace_sizes():
    lib = dion.load()
    t = lib.dion_embedding_grad_workspace_size
    assert t(0, 5, 8) == 0 and t(-1, 5, 8) == 0 and t(5, 0, 8) == 0 and t(5, 1 << 24, 8) == 0
    assert 0 < t(100, 5, 8) < t(10000, 5, 8) < t(100000, 5, 8)
    x = lib.dion_linear_xent_workspace_size
    assert x(-1, 5, 8, 0, 0, 0) == 0 and x(5, 5, 8, 2, 0, 0) == 0 and x(5, 5, 8, 0, 3, 1) == 0
    assert 0 < x(64, 32000, 2048, 1, 1, 0) < x(64, 32000, 2048, 1, 1, 1)
    # far less than the logits, whatever the vocabulary: D's pieces are bounded
    assert x(65536, 131072, 1024, 1, 1, 1) < 65536 * 131072 * 2 / 4
    assert x(8192, 131072, 4096, 0, 0, 1) < 8192 * 131072 * 4


def test_wrappers_refuse_cpu_tensors_and_wrong_types():
    ids, W = torch.zeros(3, dtype=torch.long), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        dion.embedding_(ids, W)
    with pytest.raises(ValueError, match="GPU"):
        dion.embedding_grad_(ids, torch.zeros(3, 8), W)
    with pytest.raises(ValueError, match="GPU"):
        dion.linear_cross_entropy_(torch.zeros(3, 8), W, ids)
    with pytest.raises(TypeError):
        dion.embedding_(ids, [1.0])
