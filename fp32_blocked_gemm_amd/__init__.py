"""Python binding of libog: exact and fast fp32 matrix product and NCHW
convolution, and operators around a language model's N x K weights (the
product with 4-bit weights, the product with an epilogue and its gradient, the
linear cross entropy with its gradient, the gradients' norm and clipping, the
Newton-Schulz update, the penalties on logits) on MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libog.so`` behind the C ABI of ``include/og.h``.  Torch supplies
device memory and the stream (the current torch stream of the tensors'
device).  There is no CPU path: without the built library, or off gfx950,
the calls raise.
"""
from __future__ import annotations

import array
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
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4
_ACTS = {None: ACT_NONE, "none": ACT_NONE, "relu": ACT_RELU, ACT_NONE: ACT_NONE, ACT_RELU: ACT_RELU}
_EPI_ACTS = {**_ACTS, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU,
             ACT_GELU: ACT_GELU, ACT_GELU_TANH: ACT_GELU_TANH, ACT_SILU: ACT_SILU}
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
    L.og_gemm_nt_epi.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, ctypes.c_int, _vp,
                                 _i64, _vp, _i64, _vp, _i64, _vp, _i64]
    L.og_gemm_nt_epi.restype = ctypes.c_int
    L.og_gemm_nt_epi_grad.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, ctypes.c_int, _vp, _i64,
                                      ctypes.c_int, _vp, _i64, _vp, _i64, _vp, _vp, _i64]
    L.og_gemm_nt_epi_grad.restype = ctypes.c_int
    for f in (L.og_gemm_nt_epi_workspace, L.og_gemm_nt_epi_grad_workspace):
        f.argtypes = [_i64, _i64, _i64, ctypes.c_int]
        f.restype = _i64
    L.og_grad_norm.argtypes = [_i64, _vp, _vp, _vp, _i64]
    L.og_grad_norm.restype = ctypes.c_int
    L.og_clip_grad_norm.argtypes = [_i64, _vp, ctypes.c_float, ctypes.c_float, _vp, _vp, _i64]
    L.og_clip_grad_norm.restype = ctypes.c_int
    L.og_grad_norm_workspace.argtypes = []
    L.og_grad_norm_workspace.restype = _i64
    L.og_logit_penalties.argtypes = [_i64, _i64, _vp, _i64, ctypes.c_int, _i64, _vp, _i64, _vp, _vp, _vp,
                                     _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64]
    L.og_logit_penalties.restype = ctypes.c_int
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
    ld, one = t.stride()
    if cols > 1 and one != 1:
        raise ValueError("columns must be contiguous (stride(1) == 1)")
    if rows <= 1 or cols == 0:
        return max(1, cols)
    return ld


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
    at = ts[0].get_device()  # (-1: not on a GPU)
    for t in ts:
        i = t.get_device()
        if i != at or i < 0:
            raise ValueError("tensors must be CUDA tensors" if min(i, at) < 0 else "tensors must be on one device")
    return ts[0].device


def _run(dev, call, *args):
    """Calls the library on the current stream of `dev` (which it makes the current device
    where it is not)."""
    torch = _torch()
    index = dev.index
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(dev):
            return _run(dev, call, *args)
    lib().og_set_stream(torch._C._cuda_getCurrentRawStream(index))
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
    if t.dtype != dtype or t.shape != (n,) or not t.is_contiguous():
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


def _act(act) -> int:
    if act not in _EPI_ACTS:
        raise ValueError(f"act must be None, 'relu', 'gelu', 'gelu_tanh' or 'silu', not {act!r}")
    return _EPI_ACTS[act]


def _product_shapes(A, B):
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("expected 2-D A and B")
    m, k = A.shape
    n, k2 = B.shape
    if k != k2:
        raise ValueError(f"inner sizes differ: {k} vs {k2}")
    code = _type(A, (F32, BF16, F16))
    if B.dtype != A.dtype:
        raise ValueError("A and B must have the same type")
    return m, n, k, code


def _matrix(t, rows, cols, dtype, what):
    if t.shape != (rows, cols) or t.dtype != dtype:
        raise ValueError(f"{what} must be [{rows}, {cols}] of {dtype}")


def gemm_nt_epi_workspace(m, n, k, dtype, grad=False) -> int:
    """Bytes gemm_nt_epi (grad: its gradient) needs, dtype F32, BF16 or F16."""
    f = lib().og_gemm_nt_epi_grad_workspace if grad else lib().og_gemm_nt_epi_workspace
    b = int(f(m, n, k, dtype))
    _check(min(b, 0))
    return b


def gemm_nt_epi(A, B, bias=None, act=None, residual=None, out=None, pre=None, need_pre=False, workspace=None):
    """C = act(A @ B.T + bias) + residual (og_gemm_nt_epi), B given as n x k.  A [m, k], B, bias
    [n] and residual [m, n] of one type, float32, bfloat16 or float16; act None, 'relu',
    'gelu', 'gelu_tanh' or 'silu'.  The residual may be out.  With need_pre (or a tensor pre to
    hold it) returns (C, A @ B.T + bias), which gemm_nt_epi_grad wants; else C."""
    torch = _torch()
    m, n, k, code = _product_shapes(A, B)
    act = _act(act)
    if out is None:
        out = torch.empty((m, n), dtype=A.dtype, device=A.device)
    if pre is None and need_pre:
        pre = torch.empty((m, n), dtype=A.dtype, device=A.device)
    _matrix(out, m, n, A.dtype, "out")
    given = [A, B, out]
    if bias is not None:
        _vector(bias, n, A.dtype, "bias")
        given.append(bias)
    extra = []
    for t, what in ((residual, "residual"), (pre, "pre")):
        if t is None:
            extra += [None, 0]
            continue
        _matrix(t, m, n, A.dtype, what)
        given.append(t)
        extra += [t.data_ptr(), _ld(t)]
    dev = _one_device(*given)
    size = lib().og_gemm_nt_epi_workspace(m, n, k, code)
    ws = None if size == 0 and workspace is None else _workspace(size, workspace, dev)
    _run(dev, lib().og_gemm_nt_epi, m, n, k, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B), code,
         None if bias is None else bias.data_ptr(), act, *extra, out.data_ptr(), _ld(out),
         *((None, 0) if ws is None else (ws.data_ptr(), ws.numel())))
    return out if pre is None else (out, pre)


def gemm_nt_epi_grad(dC, A, B, pre=None, act=None, need=(True, True, True), dA=None, dB=None, dbias=None,
                     workspace=None):
    """(dA, dB, dbias) of gemm_nt_epi for dC [m, n], from the `pre` it returned (not read where
    act is None); the residual's gradient is dC (og_gemm_nt_epi_grad).  need: which of the
    three are wanted; the others are None."""
    torch = _torch()
    m, n, k, code = _product_shapes(A, B)
    act = _act(act)
    _matrix(dC, m, n, A.dtype, "dC")
    if act != ACT_NONE:
        if pre is None:
            raise ValueError("the gradient of an activation needs pre")
        _matrix(pre, m, n, A.dtype, "pre")
    elif pre is not None:
        pre = None
    outs = []
    for t, shape, wanted, what in ((dA, (m, k), need[0], "dA"), (dB, (n, k), need[1], "dB"),
                                   (dbias, (n,), need[2], "dbias")):
        if not wanted:
            outs.append(None)
            continue
        if t is None:
            t = torch.empty(shape, dtype=A.dtype, device=A.device)
        if len(shape) == 1:
            _vector(t, n, A.dtype, what)
        else:
            _matrix(t, *shape, A.dtype, what)
        outs.append(t)
    dev = _one_device(dC, A, B, *([] if pre is None else [pre]), *[t for t in outs if t is not None])
    args = [p for t in outs[:2] for p in ((None, 0) if t is None else (t.data_ptr(), _ld(t)))]
    ws = _workspace(lib().og_gemm_nt_epi_grad_workspace(m, n, k, code), workspace, dev)
    _run(dev, lib().og_gemm_nt_epi_grad, m, n, k, dC.data_ptr(), _ld(dC), A.data_ptr(), _ld(A), B.data_ptr(),
         _ld(B), code, None if pre is None else pre.data_ptr(), 0 if pre is None else _ld(pre), act, *args,
         None if outs[2] is None else outs[2].data_ptr(), ws.data_ptr(), ws.numel())
    return tuple(outs)


def _dense(t) -> bool:
    """Whether the elements follow one another in memory, in whatever order of dimensions."""
    n = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != n:
            return False
        n *= size
    return True


def _run_of(t):
    """(rows, cols, row stride) of a tensor as runs of elements: one run where its elements
    follow one another in memory."""
    if t.is_contiguous() or _dense(t):
        return 1, t.numel(), t.numel()
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and t.stride(0) >= t.shape[1]:
        return t.shape[0], t.shape[1], t.stride(0)
    raise ValueError("a gradient must be dense, or 2-D with contiguous rows")


def _grads(grads, out):
    """The table of og_grad_norm's tensors, and their device."""
    torch = _torch()
    _type(grads[0], (F32, BF16, F16))
    dev = _one_device(grads[0])
    at, code_of, table = dev.index, _TYPES.get, []
    for x, y in zip(grads, grads if out is None else out):
        dtype = x.dtype
        code = code_of(dtype)
        if code is None:
            _type(x, (F32, BF16, F16))
        if x.get_device() != at or (y is not x and y.get_device() != at):
            raise ValueError("tensors must be on one device")
        if y is not x and (not y.is_same_size(x) or y.dtype != dtype):
            raise ValueError("an output must have its gradient's shape and type")
        if x.is_contiguous() and (y is x or y.is_contiguous()):
            n = x.numel()
            table += (x.data_ptr(), y.data_ptr(), 1, n, n, n, code)
            continue
        if y is x or y.stride() == x.stride():
            rows, cols, ldx = _run_of(x)
            ldy = ldx
        elif x.dim() == 2:
            rows, cols, ldx, ldy = *x.shape, _ld(x), _ld(y)
        else:
            raise ValueError("an output must have its gradient's layout")
        table += (x.data_ptr(), y.data_ptr(), rows, cols, ldx, ldy, code)
    return array.array("q", table), dev


def grad_norm(grads, workspace=None):
    """The Euclidean norm over all elements of the tensors `grads` (og_grad_norm), a tensor of
    one float32.  Types float32, bfloat16 and float16, mixed as they come; dense tensors, in
    any order of their dimensions, or 2-D ones with contiguous rows."""
    return _grad_norm(list(grads), None, None, 0.0, workspace)


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, workspace=None):
    """Scales the tensors `grads` by min(1, max_norm / (norm + eps)), norm the Euclidean norm
    over all their elements, which is returned as a tensor of one float32
    (og_clip_grad_norm).  In place, or into the tensors `out`, of the same shapes, types and
    layouts.  The host does not wait: a norm that is not finite is seen in what is returned."""
    grads = list(grads)
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("one output for each gradient expected")
    return _grad_norm(grads, out, float(max_norm), float(eps), workspace)


def _grad_norm(grads, out, max_norm, eps, workspace):
    if not grads:
        raise ValueError("at least one tensor expected")
    torch = _torch()
    L = lib()
    table, dev = _grads(grads, out)
    at = table.buffer_info()[0]
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws = _workspace(L.og_grad_norm_workspace(), workspace, dev)
    if max_norm is None:
        _run(dev, L.og_grad_norm, len(grads), at, norm.data_ptr(), ws.data_ptr(), ws.numel())
    else:
        _run(dev, L.og_clip_grad_norm, len(grads), at, max_norm, eps, norm.data_ptr(), ws.data_ptr(),
             ws.numel())
    return norm


def logit_penalties(logits, tokens=None, lengths=None, prompt_lengths=None, repetition=None,
                    frequency=None, presence=None, bias=None, mask=None, out=None):
    """Penalties for the tokens each row holds, a bias and a mask on logits [n, v] of float32,
    bfloat16 or float16 (og_logit_penalties).

    tokens [n, t] int64, of which row i's first lengths[i] count (int64; None: all), generated
    from prompt_lengths[i] on (int64; None: all were); repetition, frequency and presence [n]
    float32; bias [v], [1, v] or [n, v] float32; mask [ceil(v / 32)], [1, .] or [n, .] int32,
    bit j % 32 of word j // 32 set where token j is allowed.  What is None is left out.
    out may be logits itself."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("expected 2-D logits")
    n, v = logits.shape
    code = _type(logits, (F32, BF16, F16))
    if out is None:
        out = torch.empty((n, v), dtype=logits.dtype, device=logits.device)
    if out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out must have the logits' shape and type")
    given = [logits, out]
    t = ldt = 0
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != n or tokens.dtype != torch.int64:
            raise ValueError(f"tokens must be [{n}, t] int64")
        t, ldt = tokens.shape[1], _ld(tokens)
        given.append(tokens)
    elif not (repetition is None and frequency is None and presence is None):
        raise ValueError("a penalty without tokens")
    vectors = []
    for what, x, dtype in (("lengths", lengths, torch.int64), ("prompt_lengths", prompt_lengths, torch.int64),
                           ("repetition", repetition, torch.float32), ("frequency", frequency, torch.float32),
                           ("presence", presence, torch.float32)):
        if x is None:
            vectors.append(None)
            continue
        _vector(x, n, dtype, what)
        given.append(x)
        vectors.append(x.data_ptr())
    rows = []
    for what, x, dtype, cols in (("bias", bias, torch.float32, v), ("mask", mask, torch.int32, (v + 31) // 32)):
        if x is None:
            rows += [None, 0]
            continue
        if x.dim() == 1:
            x = x.unsqueeze(0)
        if x.dim() != 2 or x.dtype != dtype or x.shape[1] != cols or x.shape[0] not in (1, n):
            raise ValueError(f"{what} must be {dtype}, [{cols}], [1, {cols}] or [{n}, {cols}]")
        given.append(x)
        rows += [x.data_ptr(), 0 if x.shape[0] == 1 else _ld(x)]
        if x.shape[0] == 1:
            _ld(x)  # (columns contiguous)
    dev = _one_device(*given)
    _run(dev, lib().og_logit_penalties, n, v, logits.data_ptr(), _ld(logits), code, t,
         None if tokens is None else tokens.data_ptr(), ldt, *vectors, *rows, out.data_ptr(), _ld(out))
    return out
