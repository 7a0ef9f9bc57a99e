"""Argument checks of the language-model operators, on a host without a GPU:
every refusal comes before the device is touched, and empty problems are
no-ops.  No compute call is made here."""
import ctypes

import pytest

import fp32_blocked_gemm_amd as og

P = ctypes.c_void_p(256)  # non-null and aligned, never dereferenced (arguments fail first)
ODD = ctypes.c_void_p(264)
NULL = None
BIG = 1 << 60


@pytest.fixture(scope="module")
def L():
    return og.lib()


def _no_gpu():
    try:
        import torch
        if torch.cuda.is_available():
            pytest.skip("a GPU is present")
    except ImportError:
        pass


def _q4(L, m=3, n=5, k=100, A=P, type=0, lda=100, Q=P, ldq=50, S=P, stype=0, lds=4, Z=NULL, ldz=0,
        group=32, C=P, ldc=5):
    return L.og_gemm_nt_q4(m, n, k, A, type, lda, Q, ldq, S, stype, lds, Z, ldz, group, C, ldc)


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(type=-1), dict(stype=3), dict(m=-1), dict(n=-1), dict(k=-1),
    dict(group=0), dict(group=16), dict(group=48), dict(group=-32), dict(lda=99), dict(ldq=49),
    dict(lds=3), dict(Z=P, ldz=3), dict(ldc=4), dict(A=NULL), dict(Q=NULL), dict(S=NULL),
    dict(C=NULL), dict(k=0, lda=0), dict(k=101, lda=101, ldq=50),
])
def test_q4_rejects_before_launch(L, kw):
    assert _q4(L, **kw) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(m=(1 << 19) + 1), dict(n=(1 << 25) + 1, ldc=1 << 31),
                                dict(k=(1 << 28) + 1, lda=1 << 31, ldq=1 << 30, lds=1 << 30),
                                dict(m=1 << 19, n=1 << 30, ldc=1 << 30)])
def test_q4_too_large(L, kw):
    assert _q4(L, **kw) == og.OG_ERR_TOO_LARGE


def test_q4_empty_and_valid(L):
    assert _q4(L, m=0, A=NULL, C=NULL) == og.OG_OK
    assert _q4(L, n=0, Q=NULL, S=NULL, C=NULL, ldc=1) == og.OG_OK
    _no_gpu()
    assert _q4(L) == og.OG_ERR_DEVICE  # valid arguments get as far as the device check
    assert _q4(L, k=0, lda=1, ldq=1, lds=1, A=NULL, Q=NULL, S=NULL) == og.OG_ERR_DEVICE


def _ce(L, n=3, v=5, d=8, X=P, ldx=8, W=P, ldw=8, type=0, target=P, ignore=-100, loss=P, lse=P,
        ws=P, bytes=BIG):
    return L.og_linear_cross_entropy(n, v, d, X, ldx, W, ldw, type, target, ignore, loss, lse, ws, bytes)


def _ce_grad(L, n=3, v=5, d=8, X=P, ldx=8, W=P, ldw=8, type=0, target=P, ignore=-100, lse=P, dloss=P,
             dX=P, lddx=8, dW=P, lddw=8, ws=P, bytes=BIG):
    return L.og_linear_cross_entropy_grad(n, v, d, X, ldx, W, ldw, type, target, ignore, lse, dloss,
                                          dX, lddx, dW, lddw, ws, bytes)


SHARED = [dict(type=2), dict(type=-1), dict(n=-1), dict(v=0), dict(d=0), dict(ldx=7), dict(ldw=7),
          dict(X=NULL), dict(W=NULL), dict(target=NULL), dict(ws=NULL), dict(bytes=100), dict(ws=ODD)]


@pytest.mark.parametrize("kw", SHARED + [dict(loss=NULL), dict(lse=NULL)])
def test_ce_rejects_before_launch(L, kw):
    assert _ce(L, **kw) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", SHARED + [dict(lse=NULL), dict(dloss=NULL), dict(lddx=7), dict(lddw=7)])
def test_ce_grad_rejects_before_launch(L, kw):
    assert _ce_grad(L, **kw) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(n=(1 << 24) + 1), dict(v=(1 << 28) + 1),
                                dict(d=(1 << 18) + 1, ldx=1 << 19, ldw=1 << 19), dict(ldw=(1 << 22) + 1)])
def test_ce_too_large(L, kw):
    assert _ce(L, **kw) == og.OG_ERR_TOO_LARGE


def test_ce_empty_and_valid(L):
    assert _ce(L, n=0, X=NULL, W=NULL, target=NULL, loss=NULL, lse=NULL) == og.OG_OK
    assert _ce_grad(L, dX=NULL, dW=NULL) == og.OG_OK
    assert _ce_grad(L, n=0, dW=NULL) == og.OG_OK
    _no_gpu()
    assert _ce(L) == og.OG_ERR_DEVICE
    assert _ce_grad(L, dX=NULL) == og.OG_ERR_DEVICE
    # an empty batch still clears dW
    assert _ce_grad(L, n=0, X=NULL, W=NULL, target=NULL, lse=NULL, dloss=NULL) == og.OG_ERR_DEVICE


def test_ce_workspace(L):
    f = L.og_linear_cross_entropy_workspace
    assert f(3, 5, 8, 2, 0) == og.OG_ERR_INVALID_ARG
    assert f(-1, 5, 8, 0, 0) == og.OG_ERR_INVALID_ARG
    assert f(1 << 25, 5, 8, 0, 0) == og.OG_ERR_TOO_LARGE
    for n, v, d, t in ((1, 5, 8, 0), (777, 50021, 768, 0), (4096, 32768, 4096, 1)):
        # far below the logits of a large problem, and enough is accepted up to the device
        need = f(n, v, d, t, 1)
        assert 0 < need
        if n * v > 1 << 26:
            assert need < 4 * n * v
        assert _ce_grad(L, n=n, v=v, d=d, ldx=d, ldw=d, lddx=d, lddw=d, type=t,
                        bytes=need - 1) == og.OG_ERR_INVALID_ARG


def _ns(L, batch=1, m=3, n=5, G=P, ldg=5, sg=0, type=0, steps=5, a=3.4, b=-4.8, c=2.0, eps=1e-7, O=P,
        ldo=5, so=0, ws=P, bytes=BIG):
    return L.og_newton_schulz(batch, m, n, G, ldg, sg, type, steps, a, b, c, eps, O, ldo, so, ws, bytes)


@pytest.mark.parametrize("kw", [
    dict(type=2), dict(type=-1), dict(batch=-1), dict(m=-1), dict(n=-1), dict(steps=0), dict(steps=65),
    dict(a=float("nan")), dict(b=float("inf")), dict(c=float("-inf")), dict(eps=-1e-7),
    dict(eps=float("nan")), dict(ldg=4), dict(ldo=4), dict(G=NULL), dict(O=NULL), dict(ws=NULL),
    dict(bytes=100), dict(ws=ODD), dict(batch=2, sg=-15, so=15), dict(batch=2, sg=15, so=14),
    dict(a=1e4, b=0, c=0, steps=4), dict(a=1e-4, b=0, c=0, steps=3), dict(b=1e30), dict(a=4, b=2, c=3, steps=20),
])
def test_ns_rejects_before_launch(L, kw):
    assert _ns(L, **kw) == og.OG_ERR_INVALID_ARG
    assert L.og_last_error()


@pytest.mark.parametrize("kw", [dict(m=(1 << 18) + 1), dict(n=(1 << 18) + 1, ldg=1 << 19, ldo=1 << 19),
                                dict(batch=65536, sg=15, so=15)])
def test_ns_too_large(L, kw):
    assert _ns(L, **kw) == og.OG_ERR_TOO_LARGE


def test_ns_empty_and_valid(L):
    for kw in (dict(batch=0), dict(m=0), dict(n=0, ldg=1, ldo=1)):
        assert _ns(L, G=NULL, O=NULL, ws=NULL, **kw) == og.OG_OK
    assert L.og_newton_schulz_workspace(0, 3, 5, 0) == 0
    assert L.og_newton_schulz_workspace(1, 3, 5, 2) == og.OG_ERR_INVALID_ARG
    assert L.og_newton_schulz_workspace(1, 1 << 19, 5, 0) == og.OG_ERR_TOO_LARGE
    need = L.og_newton_schulz_workspace(2, 30, 50, 1)
    assert _ns(L, batch=2, m=30, n=50, ldg=50, sg=0, so=1500, ldo=50, type=1,
               bytes=need - 1) == og.OG_ERR_INVALID_ARG
    _no_gpu()
    assert _ns(L) == og.OG_ERR_DEVICE
    assert _ns(L, batch=2, sg=0, so=15) == og.OG_ERR_DEVICE  # one input for the whole batch


def test_bindings_refuse_wrong_tensors():
    torch = pytest.importorskip("torch")
    f, u, i = torch.zeros, dict(dtype=torch.uint8), dict(dtype=torch.int64)
    bad = [
        (og.gemm_nt_q4, (f(2, 64), f(3, 32, **u), f(3, 2)), dict(group=33)),
        (og.gemm_nt_q4, (f(2, 64), f(3, 31, **u), f(3, 2)), dict(group=32)),
        (og.gemm_nt_q4, (f(2, 64), f(3, 32), f(3, 2)), dict(group=32)),
        (og.gemm_nt_q4, (f(2, 64), f(3, 32, **u), f(3, 3)), dict(group=32)),
        (og.gemm_nt_q4, (f(2, 64).double(), f(3, 32, **u), f(3, 2)), dict(group=32)),
        (og.gemm_nt_q4, (f(2, 64), f(3, 32, **u), f(3, 2)), dict(group=32, zeros=f(3, 2))),
        (og.gemm_nt_q4, (f(2, 64), f(3, 32, **u), f(3, 2)), dict(group=32)),  # not on a GPU
        (og.linear_cross_entropy, (f(2, 8), f(3, 9), f(2, **i)), {}),
        (og.linear_cross_entropy, (f(2, 8), f(3, 8).bfloat16(), f(2, **i)), {}),
        (og.linear_cross_entropy, (f(2, 8).half(), f(3, 8).half(), f(2, **i)), {}),
        (og.linear_cross_entropy, (f(2, 8), f(3, 8), f(3, **i)), {}),
        (og.linear_cross_entropy, (f(2, 8), f(3, 8), f(2).int()), {}),
        (og.linear_cross_entropy, (f(2, 8), f(3, 8), f(2, **i)), {}),
        (og.linear_cross_entropy_grad, (f(2, 8), f(3, 8), f(2, **i), f(2), f(1)), {}),
        (og.linear_cross_entropy_grad, (f(2, 8), f(3, 8), f(2, **i), f(2), f(2).double()), {}),
        (og.linear_cross_entropy_grad, (f(2, 8), f(3, 8), f(2, **i), f(2), f(2)), dict(dX=f(2, 9))),
        (og.newton_schulz, (f(8),), {}),
        (og.newton_schulz, (f(8, 8).half(),), {}),
        (og.newton_schulz, (f(8, 8),), dict(out=f(8, 9))),
        (og.newton_schulz, (f(8, 8),), {}),
    ]
    for call, args, kw in bad:
        with pytest.raises(ValueError):
            call(*args, **kw)
