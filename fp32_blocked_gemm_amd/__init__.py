"""Python binding of libog: exact and fast fp32 matrix product and NCHW
convolution, and three operators around a language model's N x K weights (the
product with 4-bit weights, the linear cross entropy with its gradient, the
Newton-Schulz update) on MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libog.so`` behind the C ABI of ``include/og.h``.  Torch supplies
device memory and the stream (the current torch stream of the tensors'
device).  There is no CPU path: without the built library, or off gfx950,
the calls raise.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libog.so")

OG_OK = 0
OG_ERR_INVALID_ARG = -1
OG_ERR_NOT_EXACT = -2
OG_ERR_DEVICE = -3
OG_ERR_TOO_LARGE = -4

EXACT = 0
FAST = 1
FAST_MFMA = 2  # fast under a stated tolerance (split k, fp32 matrix cores); see og.h
F32 = 0
BF16 = 1
F16 = 2
ACT_NONE = 0
ACT_RELU = 1
_ACTS = {None: ACT_NONE, "none": ACT_NONE, "relu": ACT_RELU, ACT_NONE: ACT_NONE, ACT_RELU: ACT_RELU}
_MODES = {"exact": EXACT, "fast": FAST, "fast_mfma": FAST_MFMA, EXACT: EXACT, FAST: FAST,
          FAST_MFMA: FAST_MFMA}

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_lib = None


class OgError(RuntimeError):
    """A non-zero status from libog, with the library's own message."""

    def __init__(self, status: int, message: str):
        super().__init__(f"libog status {status}: {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libog.so.  Raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python fp32_blocked_gemm_amd/build.py` (hipcc, gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    L.og_gemm_f32.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, ctypes.c_int]
    L.og_gemm_f32.restype = ctypes.c_int
    L.og_gemm_nt_f32.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, ctypes.c_int]
    L.og_gemm_nt_f32.restype = ctypes.c_int
    L.og_conv2d_f32_ex.argtypes = [_i64] * 16 + [_vp, _vp, _vp, ctypes.c_int]
    L.og_conv2d_f32_ex.restype = ctypes.c_int
    L.og_conv2d_f32_epi.argtypes = [_i64] * 16 + [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int]
    L.og_conv2d_f32_epi.restype = ctypes.c_int
    L.og_conv2d_f32.argtypes = [_i64] * 11 + [_vp, _vp, _vp, ctypes.c_int]
    L.og_conv2d_f32.restype = ctypes.c_int
    L.og_conv2d_out_size.argtypes = [_i64] * 6
    L.og_conv2d_out_size.restype = _i64
    L.og_set_stream.argtypes = [_vp]
    L.og_set_stream.restype = ctypes.c_int
    L.og_get_stream.argtypes = []
    L.og_get_stream.restype = _vp
    L.og_set_variant.argtypes = [ctypes.c_int]
    L.og_set_variant.restype = ctypes.c_int
    L.og_get_variant.argtypes = []
    L.og_get_variant.restype = ctypes.c_int
    L.og_gemm_choice.argtypes = [_i64, _i64, _i64, ctypes.c_int]
    L.og_gemm_choice.restype = ctypes.c_int
    L.og_gemm_nt_q4.argtypes = [_i64, _i64, _i64, _vp, ctypes.c_int, _i64, _vp, _i64, _vp,
                                ctypes.c_int, _i64, _vp, _i64, _i64, _vp, _i64]
    L.og_gemm_nt_q4.restype = ctypes.c_int
    L.og_newton_schulz.argtypes = ([_i64, _i64, _i64, _vp, _i64, _i64, ctypes.c_int, ctypes.c_int]
                                   + [ctypes.c_float] * 4 + [_vp, _i64, _i64, _vp, _i64])
    L.og_newton_schulz.restype = ctypes.c_int
    L.og_newton_schulz_workspace.argtypes = [_i64, _i64, _i64, ctypes.c_int]
    L.og_newton_schulz_workspace.restype = _i64
    L.og_linear_cross_entropy.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, ctypes.c_int, _vp,
                                          _i64, _vp, _vp, _vp, _i64]
    L.og_linear_cross_entropy.restype = ctypes.c_int
    L.og_linear_cross_entropy_grad.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, ctypes.c_int,
                                               _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64]
    L.og_linear_cross_entropy_grad.restype = ctypes.c_int
    L.og_linear_cross_entropy_workspace.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int]
    L.og_linear_cross_entropy_workspace.restype = _i64
    L.og_last_error.argtypes = []
    L.og_last_error.restype = ctypes.c_char_p
    L.og_version.argtypes = []
    L.og_version.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(status: int):
    if status != OG_OK:
        raise OgError(status, lib().og_last_error().decode(errors="replace"))


def _mode(mode) -> int:
    try:
        return _MODES[mode]
    except KeyError:
        raise ValueError(f"mode must be 'exact', 'fast' or 'fast_mfma', not {mode!r}") from None


def version() -> str:
    return lib().og_version().decode()


def conv2d_out_size(size: int, k: int, stride: int, pad_before: int, pad_after: int,
                    dil: int) -> int:
    return int(lib().og_conv2d_out_size(size, k, stride, pad_before, pad_after, dil))


def set_variant(variant: int):
    """Kernel variant for this thread's later calls (0 = chosen from the shape)."""
    _check(lib().og_set_variant(variant))


def get_variant() -> int:
    return int(lib().og_get_variant())


# ---------------------------------------------------------------------------
# Raw entry points: device pointers and sizes, exactly the C ABI.
# ---------------------------------------------------------------------------

def gemm_choice(m: int, n: int, k: int, mode="fast") -> int:
    """The variant og_gemm_f32's automatic choice runs for an m x n x k
    product (n >= 2) in `mode` (og_gemm_choice)."""
    v = lib().og_gemm_choice(m, n, k, _mode(mode))
    _check(min(v, 0))
    return v


def set_stream(stream_handle: int | None):
    _check(lib().og_set_stream(stream_handle))


def gemm_f32(m, n, k, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, mode):
    _check(lib().og_gemm_f32(m, n, k, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, _mode(mode)))


def gemm_nt_f32(m, n, k, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, mode):
    _check(lib().og_gemm_nt_f32(m, n, k, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, _mode(mode)))


def conv2d_f32_ex(N, Cin, H, W, Cout, G, KH, KW, sH, sW, pT, pL, pB, pR, dH, dW, x_ptr, w_ptr,
                  y_ptr, mode):
    _check(lib().og_conv2d_f32_ex(N, Cin, H, W, Cout, G, KH, KW, sH, sW, pT, pL, pB, pR, dH, dW,
                                  x_ptr, w_ptr, y_ptr, _mode(mode)))


def conv2d_f32(N, Cin, H, W, Cout, G, KH, KW, stride, pad, dil, x_ptr, w_ptr, y_ptr, mode):
    _check(lib().og_conv2d_f32(N, Cin, H, W, Cout, G, KH, KW, stride, pad, dil, x_ptr, w_ptr,
                               y_ptr, _mode(mode)))


# ---------------------------------------------------------------------------
# Torch-tensor conveniences (still only marshalling).
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _use_stream_of(t):
    torch = _torch()
    set_stream(torch.cuda.current_stream(t.device).cuda_stream)


def _ld(t) -> int:
    """Row stride of a 2-D float32 view whose columns are contiguous.

    A view with more than one column must have stride(1) == 1, whatever its
    number of rows (a single row of a column slice is not contiguous); a
    single row's stride is never used, so it passes max(1, cols)."""
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("columns must be contiguous (stride(1) == 1)")
    if rows <= 1 or cols == 0:
        return max(1, cols)
    return t.stride(0)


def _check_f32_cuda(*ts):
    torch = _torch()
    dev = None
    for t in ts:
        if t.dtype != torch.float32 or not t.is_cuda:
            raise ValueError("tensors must be float32 CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors must be on one device")
    return dev


def gemm(A, B, mode="exact", out=None):
    """C = A @ B on 2-D float32 CUDA tensors (row strides as lda/ldb/ldc)."""
    torch = _torch()
    m, k = A.shape
    k2, n = B.shape
    if k != k2:
        raise ValueError(f"inner sizes differ: {k} vs {k2}")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    if tuple(out.shape) != (m, n):
        raise ValueError("out has the wrong shape")
    dev = _check_f32_cuda(A, B, out)
    with torch.cuda.device(dev):
        _use_stream_of(out)
        gemm_f32(m, n, k, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B), out.data_ptr(), _ld(out),
                 mode)
    return out


def gemm_nt(A, B, mode="exact", out=None):
    """C = A @ B.T on 2-D float32 CUDA tensors, B given as n x k (row strides as lda/ldb/ldc)."""
    torch = _torch()
    m, k = A.shape
    n, k2 = B.shape
    if k != k2:
        raise ValueError(f"inner sizes differ: {k} vs {k2}")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    if tuple(out.shape) != (m, n):
        raise ValueError("out has the wrong shape")
    dev = _check_f32_cuda(A, B, out)
    with torch.cuda.device(dev):
        _use_stream_of(out)
        gemm_nt_f32(m, n, k, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B), out.data_ptr(),
                    _ld(out), mode)
    return out


def conv2d(x, w, stride=(1, 1), pad=(0, 0, 0, 0), dil=(1, 1), groups=1, mode="exact",
           out=None, bias=None, act=None, residual=None):
    """NCHW convolution; pad = (top, left, bottom, right).  With bias (Cout),
    act ('relu') or residual (the output's shape) the epilogue runs in the
    same kernels: bias, then activation, then residual."""
    torch = _torch()
    if isinstance(stride, int):
        stride = (stride, stride)
    if isinstance(dil, int):
        dil = (dil, dil)
    if isinstance(pad, int):
        pad = (pad, pad, pad, pad)
    N, Cin, H, W = x.shape
    Cout, cin_g, KH, KW = w.shape
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    if cin_g * groups != Cin:
        raise ValueError(f"w.shape[1] * groups = {cin_g * groups} != Cin = {Cin}")
    OH = conv2d_out_size(H, KH, stride[0], pad[0], pad[2], dil[0])
    OW = conv2d_out_size(W, KW, stride[1], pad[1], pad[3], dil[1])
    if OH < 1 or OW < 1:
        raise ValueError("the window does not fit the padded input")
    if out is None:
        out = torch.empty((N, Cout, OH, OW), dtype=torch.float32, device=x.device)
    if tuple(out.shape) != (N, Cout, OH, OW) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [N, Cout, OH, OW] tensor")
    dev = _check_f32_cuda(x, w, out)
    if act not in _ACTS:
        raise ValueError(f"act must be None or 'relu', not {act!r}")
    if bias is not None:
        _check_f32_cuda(bias, out)
        if tuple(bias.shape) != (Cout,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous tensor of Cout floats")
    if residual is not None:
        _check_f32_cuda(residual, out)
        if tuple(residual.shape) != tuple(out.shape) or not residual.is_contiguous():
            raise ValueError("residual must be a contiguous tensor of the output's shape")
    with torch.cuda.device(dev):
        _use_stream_of(out)
        if bias is None and residual is None and _ACTS[act] == ACT_NONE:
            conv2d_f32_ex(N, Cin, H, W, Cout, groups, KH, KW, stride[0], stride[1], pad[0],
                          pad[1], pad[2], pad[3], dil[0], dil[1], x.data_ptr(), w.data_ptr(),
                          out.data_ptr(), mode)
        else:
            _check(lib().og_conv2d_f32_epi(
                N, Cin, H, W, Cout, groups, KH, KW, stride[0], stride[1], pad[0], pad[1], pad[2],
                pad[3], dil[0], dil[1], x.data_ptr(), w.data_ptr(),
                None if bias is None else bias.data_ptr(), _ACTS[act],
                None if residual is None else residual.data_ptr(), out.data_ptr(), _mode(mode)))
    return out


# ---------------------------------------------------------------------------
# Operators of language models around the N x K product.
# ---------------------------------------------------------------------------

_TYPES = {}


def _type(t, allowed=(F32, BF16)) -> int:
    if not _TYPES:
        torch = _torch()
        _TYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
    code = _TYPES.get(t.dtype)
    if code not in allowed:
        names = ", ".join(("float32", "bfloat16", "float16")[a] for a in allowed)
        raise ValueError(f"a tensor of {t.dtype}: {names} expected")
    return code


def _one_device(*ts):
    dev = ts[0].device
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        if t.device != dev:
            raise ValueError("tensors must be on one device")
    return dev


def _run(dev, call, *args):
    """Calls the library on the current stream of `dev` (which it makes the current device
    where it is not)."""
    torch = _torch()
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return _run(dev, call, *args)
    L = lib()
    L.og_set_stream(torch._C._cuda_getCurrentRawStream(dev.index))
    status = call(*args)
    if status != OG_OK:
        _check(status)


def _workspace(nbytes, workspace, dev):
    """`workspace` (a CUDA byte tensor the caller keeps), or one of the allocator's
    for this call, on the current stream."""
    torch = _torch()
    _check(min(nbytes, 0))
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the tensors' device")
    return workspace


def gemm_nt_q4(A, Q, scales, zeros=None, group=128, out=None):
    """C = A @ W.T with 4-bit weights W[j][p] = (q[j][p] - z[j][p // group]) * s[j][p // group]
    (og_gemm_nt_q4).  A [m, k] float32, bfloat16 or float16; Q [n, ceil(k / 2)] uint8, two
    codes a byte, the even k low; scales [n, ceil(k / group)] of any of the three types;
    zeros the same shape, uint8, or None for 8.  C has A's type."""
    torch = _torch()
    if A.dim() != 2 or Q.dim() != 2:
        raise ValueError("expected 2-D A and Q")
    m, k = A.shape
    n = Q.shape[0]
    if group < 32 or group % 32:
        raise ValueError("group must be a positive multiple of 32")
    groups = -(-k // group)
    every = (F32, BF16, F16)
    code, scode = _type(A, every), _type(scales, every)
    if Q.dtype != torch.uint8 or Q.shape[1] != (k + 1) // 2:
        raise ValueError(f"Q must be uint8 of {(k + 1) // 2} columns for k = {k}")
    if tuple(scales.shape) != (n, groups):
        raise ValueError(f"scales must be [{n}, {groups}]")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape):
        raise ValueError("zeros must be uint8 of the scales' shape")
    if out is None:
        out = torch.empty((m, n), dtype=A.dtype, device=A.device)
    if tuple(out.shape) != (m, n) or out.dtype != A.dtype:
        raise ValueError("out must be [m, n] of A's type")
    dev = _one_device(A, Q, scales, out, *([] if zeros is None else [zeros]))
    _run(dev, lib().og_gemm_nt_q4, m, n, k, A.data_ptr(), code, _ld(A), Q.data_ptr(), _ld(Q),
         scales.data_ptr(), scode, _ld(scales), None if zeros is None else zeros.data_ptr(),
         0 if zeros is None else _ld(zeros), group, out.data_ptr(), _ld(out))
    return out


def newton_schulz_workspace(batch, m, n, dtype) -> int:
    """Bytes newton_schulz needs for `batch` m x n matrices of `dtype` (F32 or BF16)."""
    b = int(lib().og_newton_schulz_workspace(batch, m, n, dtype))
    _check(min(b, 0))
    return b


def newton_schulz(G, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, out=None,
                  workspace=None):
    """The orthogonalised update of G (og_newton_schulz): X = G / (|G| + eps), then `steps`
    times X <- a X + (b A + c A A) X with A = X X^T and (a, b, c) = coeffs.

    G: float32 or bfloat16, [..., m, n], the last two dimensions a matrix with contiguous
    rows; any leading dimensions are a batch (a view that does not reduce to one batch
    stride is refused).  out may be G itself.  Coefficients that may lift the singular values
    past 2^37 before the last step are refused."""
    torch = _torch()
    if G.dim() < 2:
        raise ValueError("expected a tensor of at least two dimensions")
    code = _type(G)
    if out is None:
        out = torch.empty(G.shape, dtype=G.dtype, device=G.device)
    if out.shape != G.shape or out.dtype != G.dtype:
        raise ValueError("out must have G's shape and type")
    dev = _one_device(G, out)
    m, n = G.shape[-2:]
    batch = G.shape[:-2].numel()
    g3, o3 = G, out
    if G.dim() != 3:
        try:
            g3, o3 = G.view(batch, m, n), out.view(batch, m, n)
        except RuntimeError:
            raise ValueError("the leading dimensions must reduce to one batch stride") from None
    ws = _workspace(lib().og_newton_schulz_workspace(batch, m, n, code), workspace, dev)
    a, b, c = coeffs
    rows_g, rows_o = _ld(g3[0]) if batch else max(1, n), _ld(o3[0]) if batch else max(1, n)
    _run(dev, lib().og_newton_schulz, batch, m, n, g3.data_ptr(), rows_g,
         g3.stride(0) if batch > 1 else 0, code, steps, a, b, c, eps, o3.data_ptr(), rows_o,
         o3.stride(0) if batch > 1 else 0, ws.data_ptr(), ws.numel())
    return out


def _vector(t, n, dtype, what):
    if t.dtype != dtype or tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous tensor of {n} {dtype} values")


def _lce_shapes(X, W, target):
    torch = _torch()
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("expected 2-D X and W")
    n, d = X.shape
    v, d2 = W.shape
    if d != d2:
        raise ValueError(f"inner sizes differ: {d} vs {d2}")
    code = _type(X)
    if W.dtype != X.dtype:
        raise ValueError("X and W must have the same type")
    _vector(target, n, torch.int64, "target")
    return n, v, d, code


def linear_cross_entropy_workspace(n, v, d, dtype, grad=False) -> int:
    """Bytes linear_cross_entropy (grad: its gradient) needs, dtype F32 or BF16."""
    b = int(lib().og_linear_cross_entropy_workspace(n, v, d, dtype, int(bool(grad))))
    _check(min(b, 0))
    return b


def linear_cross_entropy(X, W, target, ignore_index=-100, loss=None, lse=None, workspace=None):
    """(loss, lse) of each row: the softmax cross entropy of X @ W.T against target, the
    logits never kept (og_linear_cross_entropy).  X [n, d] and W [v, d] float32 or
    bfloat16, target [n] int64; loss and lse [n] float32."""
    torch = _torch()
    n, v, d, code = _lce_shapes(X, W, target)
    loss = torch.empty(n, dtype=torch.float32, device=X.device) if loss is None else loss
    lse = torch.empty(n, dtype=torch.float32, device=X.device) if lse is None else lse
    _vector(loss, n, torch.float32, "loss")
    _vector(lse, n, torch.float32, "lse")
    dev = _one_device(X, W, target, loss, lse)
    ws = _workspace(lib().og_linear_cross_entropy_workspace(n, v, d, code, 0), workspace, dev)
    _run(dev, lib().og_linear_cross_entropy, n, v, d, X.data_ptr(), _ld(X), W.data_ptr(), _ld(W),
         code, target.data_ptr(), ignore_index, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
         ws.numel())
    return loss, lse


def linear_cross_entropy_grad(X, W, target, lse, dloss, ignore_index=-100, dX=None, dW=None,
                              need=(True, True), workspace=None):
    """(dX, dW) of linear_cross_entropy for dloss [n] float32, from the lse it returned for
    the same X, W and target (og_linear_cross_entropy_grad).  need: which of the two are
    wanted; the other is None."""
    torch = _torch()
    n, v, d, code = _lce_shapes(X, W, target)
    _vector(lse, n, torch.float32, "lse")
    _vector(dloss, n, torch.float32, "dloss")
    outs = []
    for t, like, wanted in ((dX, X, need[0]), (dW, W, need[1])):
        if wanted and t is None:
            t = torch.empty(like.shape, dtype=like.dtype, device=like.device)
        if t is not None and (t.shape != like.shape or t.dtype != like.dtype):
            raise ValueError("a gradient must have its tensor's shape and type")
        outs.append(t if wanted else None)
    given = [t for t in outs if t is not None]
    dev = _one_device(X, W, target, lse, dloss, *given)
    args = [p for t in outs for p in ((None, 0) if t is None else (t.data_ptr(), _ld(t)))]
    ws = _workspace(lib().og_linear_cross_entropy_workspace(n, v, d, code, 1), workspace, dev)
    _run(dev, lib().og_linear_cross_entropy_grad, n, v, d, X.data_ptr(), _ld(X), W.data_ptr(),
         _ld(W), code, target.data_ptr(), ignore_index, lse.data_ptr(), dloss.data_ptr(), *args,
         ws.data_ptr(), ws.numel())
    return tuple(outs)
