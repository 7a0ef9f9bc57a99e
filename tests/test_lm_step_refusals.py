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
