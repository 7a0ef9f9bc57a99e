"""Argument checks of the norm over gradients, its clipping and the penalties on logits, on a
host without a GPU: every refusal comes before the device is touched."""
import ctypes

import pytest

import fp32_blocked_gemm_amd as og
from test_lm_refusals import BIG, NULL, ODD, P, _no_gpu


@pytest.fixture(scope="module")
def L():
    return og.lib()


def _penalties(L, n=3, v=100, Z=P, ldz=100, type=0, t=8, tokens=P, ldt=8, lengths=NULL, prompts=NULL, repetition=P,
               frequency=P, presence=P, bias=P, ldb=0, mask=P, ldm=0, O=P, ldo=100):
    return L.og_logit_penalties(n, v, Z, ldz, type, t, tokens, ldt, lengths, prompts, repetition, frequency, presence,
                                bias, ldb, mask, ldm, O, ldo)


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(type=-1), dict(n=-1), dict(v=-1), dict(t=-1), dict(ldz=99), dict(ldo=99), dict(ldt=7),
    dict(t=0, ldt=0), dict(ldb=99), dict(ldb=-1), dict(ldm=3), dict(ldm=-4), dict(Z=NULL), dict(O=NULL),
    dict(tokens=NULL), dict(ldz=101), dict(v=0, ldz=0),
])
def test_penalties_reject_before_launch(L, kw):
    assert _penalties(L, **kw) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(n=(1 << 24) + 1), dict(v=(1 << 28) + 1, ldz=1 << 29, ldo=1 << 29),
                                dict(t=1 << 31, ldt=1 << 31)])
def test_penalties_too_large(L, kw):
    assert _penalties(L, **kw) == og.OG_ERR_TOO_LARGE


def test_penalties_empty_and_valid(L):
    assert _penalties(L, n=0, Z=NULL, O=NULL) == og.OG_OK
    assert _penalties(L, v=0, Z=NULL, O=NULL) == og.OG_OK
    _no_gpu()
    assert _penalties(L) == og.OG_ERR_DEVICE
    assert _penalties(L, t=0, ldt=1, tokens=NULL) == og.OG_ERR_DEVICE
    assert _penalties(L, n=1, ldz=101) == og.OG_ERR_DEVICE
    none = dict(repetition=NULL, frequency=NULL, presence=NULL, tokens=NULL)
    assert _penalties(L, bias=NULL, mask=NULL, **none) == og.OG_ERR_DEVICE


class Grad(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (name, ctypes.c_int64) for name in ("rows", "cols", "ldx", "ldy", "type")]


def _grads(*kws):
    base = dict(x=256, y=256, rows=3, cols=5, ldx=5, ldy=5, type=0)
    each = [{**base, "x": 4096 * i, "y": 4096 * i, **kw} for i, kw in enumerate(kws, 1)]
    return (Grad * len(kws))(*[Grad(**kw) for kw in each])


def _clip(L, grads, count=None, limit=1.0, eps=1e-6, norm=P, ws=P, bytes=BIG):
    return L.og_clip_grad_norm(len(grads) if count is None else count, grads, limit, eps, norm, ws, bytes)


def _norm(L, grads, count=None, norm=P, ws=P, bytes=BIG):
    return L.og_grad_norm(len(grads) if count is None else count, grads, norm, ws, bytes)


@pytest.mark.parametrize("kw", [dict(type=3), dict(type=-1), dict(rows=-1), dict(cols=-1), dict(ldx=4), dict(x=0)])
@pytest.mark.parametrize("call", [_clip, _norm])
def test_tensors_rejected_before_launch(L, call, kw):
    assert call(L, _grads({}, kw)) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(ldy=4), dict(y=0), dict(ldy=6), dict(y=4096)])
def test_outputs_rejected_before_launch(L, kw):
    assert _clip(L, _grads({}, kw)) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(count=-1), dict(norm=NULL), dict(ws=NULL), dict(ws=ODD), dict(bytes=100)])
@pytest.mark.parametrize("call", [_clip, _norm])
def test_calls_rejected_before_launch(L, call, kw):
    assert call(L, _grads({}), **kw) == og.OG_ERR_INVALID_ARG
    assert call(L, None, count=1, **{k: v for k, v in kw.items() if k != "count"}) == og.OG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(limit=-1.0), dict(limit=float("nan")), dict(limit=float("inf")), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(eps=float("inf"))])
def test_limits_rejected_before_launch(L, kw):
    assert _clip(L, _grads({}), **kw) == og.OG_ERR_INVALID_ARG


def test_too_many_or_too_large(L):
    for call in (_clip, _norm):
        assert call(L, _grads({}), count=(1 << 20) + 1) == og.OG_ERR_TOO_LARGE
        for kw in (dict(rows=1 << 21, cols=1 << 20, ldx=1 << 20, ldy=1 << 20), dict(rows=1, cols=(1 << 40) + 1),
                   dict(rows=2, cols=1 << 31, ldx=1 << 32, ldy=1 << 32)):
            assert call(L, _grads(kw)) == og.OG_ERR_TOO_LARGE, kw


def test_valid_tensors_reach_the_device(L):
    _no_gpu()
    some = _grads({}, dict(rows=0, x=0, y=0), dict(cols=0, x=0, y=0), dict(rows=1, ldx=0, ldy=0), dict(type=2))
    assert _clip(L, some) == og.OG_ERR_DEVICE and _norm(L, some) == og.OG_ERR_DEVICE
    assert _norm(L, _grads(dict(y=0, ldy=0))) == og.OG_ERR_DEVICE
    assert _clip(L, _grads(dict(x=8192, ldy=9))) == og.OG_ERR_DEVICE
    assert _clip(L, None, count=0) == og.OG_ERR_DEVICE  # the norm of nothing is written there


def _epi(L, m=3, n=5, k=8, A=P, lda=8, W=P, ldw=8, type=0, bias=P, act=2, R=P, ldr=5, Pre=ODD, ldp=5, C=P, ldc=5, ws=P,
         bytes=BIG):
    return L.og_gemm_nt_epi(m, n, k, A, lda, W, ldw, type, bias, act, R, ldr, Pre, ldp, C, ldc, ws, bytes)


def _epi_grad(L, m=3, n=5, k=8, dC=P, lddc=5, A=P, lda=8, W=P, ldw=8, type=0, Pre=P, ldp=5, act=2, dA=P, ldda=8, dW=P,
              lddw=8, dbias=P, ws=P, bytes=BIG):
    return L.og_gemm_nt_epi_grad(m, n, k, dC, lddc, A, lda, W, ldw, type, Pre, ldp, act, dA, ldda, dW, lddw, dbias, ws,
                                 bytes)


SHARED = [dict(type=3), dict(type=-1), dict(act=5), dict(act=-1), dict(m=-1), dict(n=-1), dict(k=-1), dict(lda=7),
          dict(ldw=7), dict(ldp=4), dict(A=NULL), dict(W=NULL), dict(ws=ODD),
          dict(ws=NULL, m=900, n=900, k=900, **dict.fromkeys(("lda", "ldw", "ldr", "ldp", "ldc", "lddc", "ldda", "lddw"),
                                                             900))]


def _given(call, kw):
    import inspect
    return {k: v for k, v in kw.items() if k in inspect.signature(call).parameters}


@pytest.mark.parametrize("kw", SHARED + [dict(ldr=4), dict(ldc=4), dict(C=NULL), dict(ldr=6), dict(Pre=P), dict(k=0, lda=0)])
def test_epi_rejects_before_launch(L, kw):
    assert _epi(L, **_given(_epi, kw)) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", SHARED + [dict(lddc=4), dict(ldda=7), dict(lddw=7), dict(dC=NULL), dict(Pre=NULL)])
def test_epi_grad_rejects_before_launch(L, kw):
    assert _epi_grad(L, **_given(_epi_grad, kw)) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(m=(1 << 24) + 1), dict(n=(1 << 20) + 1), dict(k=(1 << 20) + 1),
                                dict(m=1 << 24, n=1 << 13), dict(n=1 << 20, k=1 << 17), dict(m=1 << 24, k=1 << 13)])
@pytest.mark.parametrize("call", [_epi, _epi_grad])
def test_epi_too_large(L, call, kw):
    every = dict.fromkeys(("lda", "ldw", "ldr", "ldp", "ldc", "lddc", "ldda", "lddw"), 1 << 21)
    assert call(L, **_given(call, {**every, **kw})) == og.OG_ERR_TOO_LARGE


def test_epi_empty_and_valid(L):
    assert _epi(L, m=0, A=NULL, C=NULL, ws=NULL, bytes=0) == og.OG_OK
    assert _epi(L, n=0, W=NULL, C=NULL, ws=NULL, bytes=0) == og.OG_OK
    assert _epi_grad(L, dA=NULL, dW=NULL, dbias=NULL) == og.OG_OK
    assert _epi_grad(L, k=0, lda=1, ldw=1, ldda=1, lddw=1, dbias=NULL) == og.OG_OK
    assert _epi_grad(L, m=0, dW=NULL, dbias=NULL) == og.OG_OK
    _no_gpu()
    for type in (0, 1, 2):
        assert _epi(L, type=type) == og.OG_ERR_DEVICE
        assert _epi(L, type=type, k=0, lda=1, ldw=1, A=NULL, W=NULL) == og.OG_ERR_DEVICE
        assert _epi_grad(L, type=type) == og.OG_ERR_DEVICE
        assert _epi_grad(L, type=type, Pre=NULL, ldp=0, act=0) == og.OG_ERR_DEVICE
        # without dW, A is not wanted; without dA, W is not
        assert _epi_grad(L, type=type, A=NULL, lda=0, dW=NULL, lddw=0) == og.OG_ERR_DEVICE
        assert _epi_grad(L, type=type, W=NULL, ldw=0, dA=NULL, ldda=0) == og.OG_ERR_DEVICE
        # an empty batch clears dW and dbias
        assert _epi_grad(L, type=type, m=0, dC=NULL, A=NULL, W=NULL, Pre=NULL) == og.OG_ERR_DEVICE


def test_epi_workspace(L):
    for f in (L.og_gemm_nt_epi_workspace, L.og_gemm_nt_epi_grad_workspace):
        assert f(3, 5, 8, 3) == og.OG_ERR_INVALID_ARG
        assert f(-1, 5, 8, 0) == og.OG_ERR_INVALID_ARG
        assert f(1 << 25, 5, 8, 0) == og.OG_ERR_TOO_LARGE
    for type in (0, 1, 2):
        m, n, k = 1300, 800, 512
        need = L.og_gemm_nt_epi_grad_workspace(m, n, k, type)
        strides = dict(lddc=n, lda=k, ldw=k, ldp=n, ldda=k, lddw=k)
        assert _epi_grad(L, m, n, k, type=type, bytes=need - 1, **strides) == og.OG_ERR_INVALID_ARG
        need = L.og_gemm_nt_epi_workspace(m, n, k, type)
        strides = dict(lda=k, ldw=k, ldr=n, ldp=n, ldc=n)
        assert _epi(L, m, n, k, type=type, bytes=need - 1, **strides) == og.OG_ERR_INVALID_ARG
