"""Python binding for libforge.so: the fused weight-gradient GEMM + optimizer.

Thin ctypes marshalling over the C ABI declared in ``include/forge.h``; the
functions carry the same names.  Tensors are torch CUDA tensors; sizes are
taken from their shapes, pointers from ``data_ptr()`` and the stream from the
current torch stream unless one is given.  Every step of the computation runs
in the library's CUDA kernels: there is no CPU or PyTorch fallback, and
importing a function fails loudly if ``libforge.so`` has not been built
(``python -m weight_grad_gemm_gb300.build``).

Layouts: X [K, N] (tokens x d_in), dY [K, M] (tokens x d_out), W / m / v /
dW [N, M] (d_in x d_out), all contiguous; grouped: W / m / v [E, N, M] and
int32 offsets [E+1] on the device.
"""
from __future__ import annotations

import ctypes
import math
import os
from array import array
from operator import attrgetter

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libforge.so")

FORGE_OK = 0
FORGE_ERR_INVALID_ARG = -1
FORGE_ERR_UNSUPPORTED_DTYPE = -2
FORGE_ERR_UNSUPPORTED_DEVICE = -3
FORGE_ERR_MISALIGNED = -4
FORGE_ERR_CUDA = -5
FORGE_ERR_TIMEOUT = -6
FORGE_ERR_SCRATCH_TOO_SMALL = -7

FORGE_BF16 = 0
FORGE_E4M3 = 1
FORGE_F32 = 2
FORGE_I32 = 3
FORGE_I64 = 4

EXPORTS = ("forge_wgrad_adamw", "forge_wgrad_adamw_noalloc", "forge_wgrad_adamw_multi",
           "forge_wgrad_sgdm", "forge_wgrad_only",
           "forge_quantize_e4m3", "forge_dgrad", "forge_backward_adamw",
           "forge_grouped_wgrad_adamw", "forge_owner_adamw", "forge_owner_sgdm",
           "forge_token_logprob", "forge_token_logprob_grad", "forge_embedding",
           "forge_embedding_grad", "forge_embedding_adamw", "forge_grad_norm", "forge_clip_grads",
           "forge_layer_norm", "forge_layer_norm_grad", "forge_moe_route", "forge_moe_route_grad",
           "forge_quantize_e4m3_blocks", "forge_linear_e4m3", "forge_grouped_linear_e4m3",
           "forge_status_string", "forge_get_device_status",
           "forge_selftest_wait_timeout", "forge_version")


class ForgeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {forge_status_string(status)} ({status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libforge.so with argument types set (raw C calls)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -m weight_grad_gemm_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, F, I = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                         ctypes.c_int)
    L.forge_wgrad_adamw.argtypes = [P, P, P, P, P, I64, I64, I64, I, I, F, F, F, F, F, I64, P, P]
    L.forge_wgrad_adamw_noalloc.argtypes = L.forge_wgrad_adamw.argtypes
    L.forge_wgrad_adamw_multi.argtypes = [P, I64, I64, I32, P, P, P, P, P, I, I, F, F, F, F, F,
                                          I64, P]
    L.forge_quantize_e4m3.argtypes = [P, I, I64, P, P, P]
    L.forge_dgrad.argtypes = [P, P, P, I64, I64, I64, I, P]
    L.forge_backward_adamw.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I, I, F, F, F, F, F,
                                       I64, P]
    L.forge_wgrad_sgdm.argtypes = [P, P, P, P, I64, I64, I64, I, I, F, F, F, P, P]
    L.forge_wgrad_only.argtypes = [P, P, P, I64, I64, I64, I, P, P]
    L.forge_grouped_wgrad_adamw.argtypes = [P, P, P, P, P, P, I32, I64, I64, I64, I, I, F, F, F,
                                            F, F, I64, P, P]
    L.forge_owner_adamw.argtypes = [P, P, P, P, I64, I, F, F, F, F, F, I64, P]
    L.forge_owner_sgdm.argtypes = [P, P, P, I64, I, F, F, F, P]
    L.forge_token_logprob.argtypes = [P, I, I64, I64, I64, P, I, F, P, P, P, I32, P, P, P]
    L.forge_token_logprob_grad.argtypes = [P, I, I64, I64, I64, P, I, F, P, P, P, P, P, I, I64, P]
    L.forge_embedding.argtypes = [P, I, I64, P, I, I64, I64, F, P, I, P]
    L.forge_embedding_grad.argtypes = [P, I, P, I, I64, I64, I64, F, P, I32, P]
    L.forge_embedding_adamw.argtypes = [P, I, P, I, I64, I64, I64, F, P, P, P, I, F, F, F, F, F,
                                        I64, P]
    L.forge_grad_norm.argtypes = [P, P, I32, I, P, P]
    L.forge_clip_grads.argtypes = [P, P, I32, I, P, F, P, I, P]
    L.forge_layer_norm.argtypes = [P, I, I64, P, P, I64, I64, F, P, I, I64, P, P, P]
    L.forge_layer_norm_grad.argtypes = [P, I, I64, P, I, I64, P, P, P, I64, I64, P, I, I64, P, P,
                                        I32, P]
    L.forge_moe_route.argtypes = [P, I, I64, I32, I64, I32, I32, P, P, P, P, P, P, P, P, P]
    L.forge_moe_route_grad.argtypes = [P, I, I64, I32, I64, I32, I32, P, P, P, P, P, P, I, I64, P]
    L.forge_quantize_e4m3_blocks.argtypes = [P, I, I64, I64, I64, I64, I32, P, P, P]
    L.forge_linear_e4m3.argtypes = [P, P, P, P, P, I, I64, I64, I64, I32, P]
    L.forge_grouped_linear_e4m3.argtypes = [P, P, P, P, P, I32, P, I, I64, I64, I64, I32, P]
    for f in ("forge_layer_norm", "forge_layer_norm_grad", "forge_moe_route",
              "forge_moe_route_grad", "forge_quantize_e4m3_blocks", "forge_linear_e4m3",
              "forge_grouped_linear_e4m3",
              "forge_token_logprob", "forge_token_logprob_grad", "forge_embedding",
              "forge_embedding_grad", "forge_embedding_adamw", "forge_grad_norm",
              "forge_clip_grads",
              "forge_wgrad_adamw", "forge_wgrad_adamw_noalloc", "forge_wgrad_adamw_multi",
              "forge_wgrad_sgdm",
              "forge_wgrad_only", "forge_quantize_e4m3", "forge_dgrad", "forge_backward_adamw",
              "forge_grouped_wgrad_adamw", "forge_owner_adamw", "forge_owner_sgdm",
              "forge_get_device_status",
              "forge_selftest_wait_timeout"):
        getattr(L, f).restype = I
    L.forge_status_string.argtypes = [I]
    L.forge_status_string.restype = ctypes.c_char_p
    L.forge_get_device_status.argtypes = []
    L.forge_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P]
    L.forge_version.argtypes = []
    L.forge_version.restype = I32
    _lib = L
    return L


# ---- marshalling helpers ---------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FORGE_BF16
    if t.dtype == torch.float8_e4m3fn:
        return FORGE_E4M3
    if t.dtype == torch.float32:
        return FORGE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


_current_stream = None  # device index -> the current stream's handle, found on first use


def _find_current_stream():
    """PyTorch's own accessor, without a Stream object around the handle (0.2
    instead of 2 us a call), or the public one where a PyTorch lacks it."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream


def _stream(stream, like):
    global _current_stream
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _current_stream is None:
        _current_stream = _find_current_stream()
    return _current_stream(like.device.index)


def _check(status: int, where: str):
    if status != FORGE_OK:
        raise ForgeError(status, where)


def _sizes(X, dY):
    if X.dim() != 2 or dY.dim() != 2 or X.shape[0] != dY.shape[0]:
        raise ValueError(f"X [K, N] and dY [K, M] expected, got {tuple(X.shape)}, {tuple(dY.shape)}")
    return dY.shape[1], X.shape[1], X.shape[0]  # M, N, K


def _scales_ptr(scales, X):
    if scales is None:
        return None
    import torch
    if scales.dtype != torch.float32 or scales.numel() != 2:
        raise ValueError("scales must be a float32 tensor [sX, sdY]")
    return _ptr(scales)


# ---- the C ABI, tensor form ------------------------------------------------

def _adamw_call(name, X, dY, W, m, v, lr, beta1, beta2, eps, wd, step, scales, stream):
    M, N, K = _sizes(X, dY)
    for t in (W, m, v):
        if tuple(t.shape) != (N, M):
            raise ValueError(f"W/m/v must be [N={N}, M={M}], got {tuple(t.shape)}")
    if m.dtype != v.dtype:
        raise TypeError("m and v must share a dtype")
    s = getattr(lib(), name)(_ptr(X), _ptr(dY), _ptr(W), _ptr(m), _ptr(v), M, N, K,
                             _dtype_code(X), _dtype_code(m), lr, beta1, beta2, eps, wd,
                             int(step), _scales_ptr(scales, X), _stream(stream, W))
    _check(s, name)


def forge_wgrad_adamw(X, dY, W, m, v, *, lr, beta1, beta2, eps, wd, step, scales=None,
                      stream=None):
    _adamw_call("forge_wgrad_adamw", X, dY, W, m, v, lr, beta1, beta2, eps, wd, step, scales,
                stream)


def forge_wgrad_adamw_noalloc(X, dY, W, m, v, *, lr, beta1, beta2, eps, wd, step, scales=None,
                              stream=None):
    """forge_wgrad_adamw staging misaligned operands into the library's fixed
    per-device buffer instead of allocating (see include/forge.h)."""
    _adamw_call("forge_wgrad_adamw_noalloc", X, dY, W, m, v, lr, beta1, beta2, eps, wd, step,
                scales, stream)


def forge_wgrad_adamw_multi(X, dYs, Ws, ms, vs, *, lr, beta1, beta2, eps, wd, step,
                            stream=None):
    """One launch of forge_wgrad_adamw for each (dY, W, m, v) of the lists, all
    with the same X (see include/forge.h)."""
    n = len(dYs)
    if not (len(Ws) == len(ms) == len(vs) == n):
        raise ValueError("dYs, Ws, ms, vs must have one entry per problem")
    sizes = [_sizes(X, d) for d in dYs]
    N, K = X.shape[1], X.shape[0]
    for (M, _, _), W, m, v in zip(sizes, Ws, ms, vs):
        for t in (W, m, v):
            if tuple(t.shape) != (N, M):
                raise ValueError(f"W/m/v must be [N={N}, M={M}], got {tuple(t.shape)}")
        if m.dtype != v.dtype or m.dtype != ms[0].dtype:
            raise TypeError("every m and v must share one dtype")
        if X.dtype != dYs[0].dtype:
            raise TypeError("X and every dY must share one dtype")
    arr = ctypes.c_void_p * max(n, 1)
    dptr = arr(*[_ptr(d).value for d in dYs])
    wptr = arr(*[_ptr(t).value for t in Ws])
    mptr = arr(*[_ptr(t).value for t in ms])
    vptr = arr(*[_ptr(t).value for t in vs])
    mlen = (ctypes.c_int64 * max(n, 1))(*[M for M, _, _ in sizes])
    s = lib().forge_wgrad_adamw_multi(_ptr(X), N, K, n, dptr, mlen, wptr, mptr, vptr,
                                      _dtype_code(X), _dtype_code(ms[0]), lr, beta1, beta2, eps,
                                      wd, int(step), _stream(stream, Ws[0]))
    _check(s, "forge_wgrad_adamw_multi")


def forge_wgrad_sgdm(X, dY, W, mom, *, lr, momentum, wd, scales=None, stream=None):
    M, N, K = _sizes(X, dY)
    for t in (W, mom):
        if tuple(t.shape) != (N, M):
            raise ValueError(f"W/mom must be [N={N}, M={M}], got {tuple(t.shape)}")
    s = lib().forge_wgrad_sgdm(_ptr(X), _ptr(dY), _ptr(W), _ptr(mom), M, N, K, _dtype_code(X),
                               _dtype_code(mom), lr, momentum, wd, _scales_ptr(scales, X),
                               _stream(stream, W))
    _check(s, "forge_wgrad_sgdm")


def forge_wgrad_only(X, dY, dW, *, scales=None, stream=None):
    M, N, K = _sizes(X, dY)
    if tuple(dW.shape) != (N, M):
        raise ValueError(f"dW must be [N={N}, M={M}], got {tuple(dW.shape)}")
    s = lib().forge_wgrad_only(_ptr(X), _ptr(dY), _ptr(dW), M, N, K, _dtype_code(X),
                               _scales_ptr(scales, X), _stream(stream, dW))
    _check(s, "forge_wgrad_only")


def forge_quantize_e4m3(x, codes, scale, *, stream=None):
    """codes (uint8 or float8_e4m3fn, x.numel() elements) and scale (float32
    [1]) from x (float32 or bfloat16): s = amax / 448, codes = nearest e4m3 of
    x / s."""
    import torch
    if codes.numel() != x.numel() or codes.element_size() != 1:
        raise ValueError("codes must hold one byte per element of x")
    if scale.dtype != torch.float32 or scale.numel() != 1:
        raise ValueError("scale must be a float32 tensor of one element")
    s = lib().forge_quantize_e4m3(_ptr(x), _dtype_code(x), x.numel(), _ptr(codes), _ptr(scale),
                                  _stream(stream, codes))
    _check(s, "forge_quantize_e4m3")


def forge_dgrad(dY, Wb, dX, *, stream=None):
    """dX [K, N] (bf16) = dY [K, M] (bf16) times Wb [N, M] (bf16) transposed."""
    K, M = dY.shape
    N = Wb.shape[0]
    if Wb.dim() != 2 or Wb.shape[1] != M or tuple(dX.shape) != (K, N):
        raise ValueError(f"dY [K, M], Wb [N, M], dX [K, N] expected, got {tuple(dY.shape)}, "
                         f"{tuple(Wb.shape)}, {tuple(dX.shape)}")
    s = lib().forge_dgrad(_ptr(dY), _ptr(Wb), _ptr(dX), M, N, K, _dtype_code(dY),
                          _stream(stream, dX))
    _check(s, "forge_dgrad")


def forge_backward_adamw(X, dY, W, m, v, dX, *, lr, beta1, beta2, eps, wd, step, Wb=None,
                         stream=None):
    """dX = dY Wb^T, then the fused dW + AdamW on W, m, v, in that order on one
    stream.  Wb: the bf16 copy of W the forward used, or None to have W
    rounded to bf16 first."""
    M, N, K = _sizes(X, dY)
    for t in (W, m, v):
        if tuple(t.shape) != (N, M):
            raise ValueError(f"W/m/v must be [N={N}, M={M}], got {tuple(t.shape)}")
    if tuple(dX.shape) != (K, N) or (Wb is not None and tuple(Wb.shape) != (N, M)):
        raise ValueError("dX must be [K, N] and Wb [N, M]")
    if m.dtype != v.dtype:
        raise TypeError("m and v must share a dtype")
    s = lib().forge_backward_adamw(_ptr(X), _ptr(dY), _ptr(W), _ptr(m), _ptr(v), _ptr(Wb),
                                   _ptr(dX), M, N, K, _dtype_code(X), _dtype_code(m), lr, beta1,
                                   beta2, eps, wd, int(step), _stream(stream, W))
    _check(s, "forge_backward_adamw")


def forge_grouped_wgrad_adamw(X, dY, W, m, v, offsets, *, lr, beta1, beta2, eps, wd, step,
                              scales=None, stream=None):
    import torch
    M, N, T = _sizes(X, dY)
    E = offsets.numel() - 1
    if offsets.dtype != torch.int32 or E < 1:
        raise ValueError("offsets must be int32 [E+1] with E >= 1")
    for t in (W, m, v):
        if tuple(t.shape) != (E, N, M):
            raise ValueError(f"W/m/v must be [E={E}, N={N}, M={M}], got {tuple(t.shape)}")
    s = lib().forge_grouped_wgrad_adamw(_ptr(X), _ptr(dY), _ptr(W), _ptr(m), _ptr(v),
                                        _ptr(offsets), E, T, M, N, _dtype_code(X),
                                        _dtype_code(m), lr, beta1, beta2, eps, wd, int(step),
                                        _scales_ptr(scales, X), _stream(stream, W))
    _check(s, "forge_grouped_wgrad_adamw")


def _same_numel(G, *ts):
    for t in ts:
        if t.numel() != G.numel():
            raise ValueError(f"gradient shard and state must have one element each, got "
                             f"{G.numel()} and {t.numel()}")


def forge_owner_adamw(G, W, m, v, *, lr, beta1, beta2, eps, wd, step, stream=None):
    """The owner's AdamW step on its shard: G (fp32, the reduce-scattered sum
    of the ranks' partial dW), W (fp32), m, v (fp32 or bf16), all of one
    shape, updated in place (see include/forge.h)."""
    import torch
    _same_numel(G, W, m, v)
    if G.dtype != torch.float32 or W.dtype != torch.float32 or m.dtype != v.dtype:
        raise TypeError("G and W must be float32, m and v one dtype")
    s = lib().forge_owner_adamw(_ptr(G), _ptr(W), _ptr(m), _ptr(v), G.numel(), _dtype_code(m),
                                lr, beta1, beta2, eps, wd, int(step), _stream(stream, W))
    _check(s, "forge_owner_adamw")


def forge_owner_sgdm(G, W, mom, *, lr, momentum, wd, stream=None):
    """The owner's SGD-momentum step on its shard (see forge_owner_adamw)."""
    import torch
    _same_numel(G, W, mom)
    if G.dtype != torch.float32 or W.dtype != torch.float32:
        raise TypeError("G and W must be float32")
    s = lib().forge_owner_sgdm(_ptr(G), _ptr(W), _ptr(mom), G.numel(), _dtype_code(mom), lr,
                               momentum, wd, _stream(stream, W))
    _check(s, "forge_owner_sgdm")


_codes = {}  # torch dtype -> forge_dtype, filled on first use


def _all_codes():
    import torch
    _codes.update({torch.bfloat16: FORGE_BF16, torch.float32: FORGE_F32,
                   torch.int32: FORGE_I32, torch.int64: FORGE_I64})
    return _codes


def _code(t, allowed, what) -> int:
    code = (_codes or _all_codes()).get(t.dtype)
    if code not in allowed:
        raise TypeError(f"{what}, got {t.dtype}")
    return code


def _id_code(t) -> int:
    return _code(t, (FORGE_I32, FORGE_I64), "token ids must be int32 or int64")


def _float_code(t) -> int:
    return _code(t, (FORGE_BF16, FORGE_F32), "bfloat16 or float32 expected")


def _rows(t, what):
    """Address, row stride, rows and columns of a 2-D tensor whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what} must be [R, V] with contiguous rows")
    R, V = shape
    ld = strides[0] if R > 1 else V
    if ld < V:
        raise ValueError(f"the rows of {what} overlap")
    return t.data_ptr(), ld, R, V


def _vector(t, n, what):
    """Pointer of an fp32 tensor of n elements, or None."""
    if t is None:
        return None
    if (_codes or _all_codes()).get(t.dtype) == FORGE_F32 and t.numel() == n and t.is_cuda and \
            t.is_contiguous():
        return t.data_ptr()
    if t.numel() != n or _float_code(t) != FORGE_F32:
        raise ValueError(f"{what} must be float32 with {n} elements")
    return _ptr(t)


def forge_token_logprob(logits, targets, logprob, *, lse=None, entropy=None, top_index=None,
                        top_logprob=None, scale=1.0, stream=None):
    """logprob [R] of the target tokens under logits [R, V] (bf16 or fp32, rows
    of any stride), and where given lse [R], entropy [R] and the k best
    entries top_index [R, k] (int32), top_logprob [R, k] of each row.  targets
    [R] int32 or int64, negative for padding; logprob and targets may both be
    None (see include/forge.h)."""
    lp, ld, R, V = _rows(logits, "logits")
    if targets is not None and targets.numel() != R:
        raise ValueError(f"targets must have {R} elements")
    k = 0
    if (top_index is None) != (top_logprob is None):
        raise ValueError("top_index and top_logprob go together")
    if top_index is not None:
        k = top_index.shape[-1]
        if tuple(top_index.shape) != (R, k) or tuple(top_logprob.shape) != (R, k):
            raise ValueError(f"top_index and top_logprob must be [R={R}, k]")
        if _id_code(top_index) != FORGE_I32 or _float_code(top_logprob) != FORGE_F32:
            raise TypeError("top_index must be int32 and top_logprob float32")
    s = lib().forge_token_logprob(lp, _float_code(logits), R, V, ld, _ptr(targets),
                                  FORGE_I32 if targets is None else _id_code(targets), scale,
                                  _vector(logprob, R, "logprob"), _vector(lse, R, "lse"),
                                  _vector(entropy, R, "entropy"), k, _ptr(top_index),
                                  _ptr(top_logprob), _stream(stream, logits))
    _check(s, "forge_token_logprob")


def forge_token_logprob_grad(logits, targets, lse, grad_logprob, dlogits, *, entropy=None,
                             grad_entropy=None, scale=1.0, stream=None):
    """dlogits [R, V] (bf16 or fp32, rows of any stride; may be logits itself)
    of sum(grad_logprob * logprob + grad_entropy * entropy), from the lse and
    entropy that forge_token_logprob gave."""
    lp, ld, R, V = _rows(logits, "logits")
    dp, ldo, *out = _rows(dlogits, "dlogits")
    if out != [R, V] or targets.numel() != R:
        raise ValueError(f"dlogits must be [R={R}, V={V}] and targets [R]")
    s = lib().forge_token_logprob_grad(lp, _float_code(logits), R, V, ld, _ptr(targets),
                                       _id_code(targets), scale, _vector(lse, R, "lse"),
                                       _vector(grad_logprob, R, "grad_logprob"),
                                       _vector(entropy, R, "entropy"),
                                       _vector(grad_entropy, R, "grad_entropy"), dp,
                                       _float_code(dlogits), ldo, _stream(stream, logits))
    _check(s, "forge_token_logprob_grad")


def _embedding_sizes(ids, rows, V_D):
    if len(V_D) != 2 or rows.dim() != 2 or tuple(rows.shape) != (ids.numel(), V_D[1]):
        raise ValueError(f"ids of T elements, [T, D] and [V, D] expected, got {tuple(ids.shape)}, "
                         f"{tuple(rows.shape)}, {tuple(V_D)}")
    return ids.numel(), V_D[0], V_D[1]


def forge_embedding(ids, W, Y, *, scale=1.0, stream=None):
    """Y [T, D] = scale * W[ids] for ids of T elements (int32 or int64, negative
    for padding: a zero row) and W [V, D]; W and Y bf16 or fp32 each."""
    T, V, D = _embedding_sizes(ids, Y, W.shape)
    s = lib().forge_embedding(_ptr(ids), _id_code(ids), T, _ptr(W), _float_code(W), V, D, scale,
                              _ptr(Y), _float_code(Y), _stream(stream, Y))
    _check(s, "forge_embedding")


def forge_embedding_grad(dY, ids, dW, *, scale=1.0, accumulate=False, stream=None):
    """dW [V, D] (fp32) = scale * the sum of dY [T, D] (bf16 or fp32) by ids, or
    that added to dW (accumulate)."""
    T, V, D = _embedding_sizes(ids, dY, dW.shape)
    if _float_code(dW) != FORGE_F32:
        raise TypeError("dW must be float32")
    s = lib().forge_embedding_grad(_ptr(dY), _float_code(dY), _ptr(ids), _id_code(ids), T, V, D,
                                   scale, _ptr(dW), int(bool(accumulate)), _stream(stream, dW))
    _check(s, "forge_embedding_grad")


def forge_embedding_adamw(dY, ids, W, m, v, *, lr, beta1, beta2, eps, wd, step, scale=1.0,
                          stream=None):
    """The sum of dY [T, D] by ids as the gradient of one AdamW step on W (fp32),
    m, v (fp32 or bf16), all [V, D], in one pass over them."""
    T, V, D = _embedding_sizes(ids, dY, W.shape)
    if tuple(m.shape) != (V, D) or tuple(v.shape) != (V, D):
        raise ValueError(f"W/m/v must be [V={V}, D={D}]")
    if _float_code(W) != FORGE_F32 or m.dtype != v.dtype:
        raise TypeError("W must be float32, m and v one dtype")
    s = lib().forge_embedding_adamw(_ptr(dY), _float_code(dY), _ptr(ids), _id_code(ids), T, V, D,
                                    scale, _ptr(W), _ptr(m), _ptr(v), _float_code(m), lr, beta1,
                                    beta2, eps, wd, int(step), _stream(stream, W))
    _check(s, "forge_embedding_adamw")


def _tensor_list(ts, what):
    """Pointers, element counts and the common dtype of a list of tensors."""
    import torch
    T = torch.Tensor
    if len(set(map(attrgetter("dtype"), ts))) > 1:
        raise TypeError(f"{what} must share one dtype")
    if not (all(map(attrgetter("is_cuda"), ts)) and all(map(T.is_contiguous, ts))):
        raise ValueError(f"{what} must be contiguous CUDA tensors")
    ptrs = array("q", map(T.data_ptr, ts))
    sizes = array("q", map(T.numel, ts))
    return ptrs, sizes, FORGE_F32 if not ts else _float_code(ts[0])


def _address(a):
    """The host address of an array; the caller holds the array during the call."""
    return a.buffer_info()[0] or None


def forge_grad_norm(grads, norm, *, stream=None):
    """norm (fp32 [1]) = the square root of the sum of squares over all tensors
    of grads (a list, bf16 or fp32)."""
    ptrs, sizes, code = _tensor_list(grads, "grads")
    s = lib().forge_grad_norm(_address(ptrs), _address(sizes), len(grads), code, _vector(norm, 1, "norm"),
                              _stream(stream, norm))
    _check(s, "forge_grad_norm")


def forge_clip_grads(grads, norm, out=None, *, max_norm, stream=None):
    """out[j] = grads[j] * min(1, max_norm / (norm + 1e-6)); in place without
    out, whose tensors may be of the other dtype (bf16 or fp32)."""
    ptrs, sizes, code = _tensor_list(grads, "grads")
    optrs, ocode = ptrs, code
    if out is not None:
        optrs, osizes, ocode = _tensor_list(out, "out")
        if len(out) != len(grads) or osizes != sizes:
            raise ValueError("out must have one tensor of the same size for each of grads")
    s = lib().forge_clip_grads(_address(ptrs), _address(sizes), len(grads), code,
                               _vector(norm, 1, "norm"), max_norm, _address(optrs), ocode, _stream(stream, norm))
    _check(s, "forge_clip_grads")


def forge_layer_norm(x, weight, bias, y, *, mean=None, rstd=None, eps=1e-5, stream=None):
    """y [R, D] = (x - mean) * rstd * weight + bias over the rows of x [R, D] (bf16
    or fp32 each, rows of any stride; y may be x itself); weight and bias (or
    None) fp32 [D].  mean and rstd [R] (fp32) are kept where given."""
    xp, ldx, R, D = _rows(x, "x")
    yp, ldy, *out = _rows(y, "y")
    if out != [R, D]:
        raise ValueError(f"y must be [R={R}, D={D}]")
    s = lib().forge_layer_norm(xp, _float_code(x), ldx, _vector(weight, D, "weight"),
                               _vector(bias, D, "bias"), R, D, eps, yp, _float_code(y), ldy,
                               _vector(mean, R, "mean"), _vector(rstd, R, "rstd"),
                               _stream(stream, x))
    _check(s, "forge_layer_norm")


def forge_layer_norm_grad(dy, x, weight, mean, rstd, dx, dweight, dbias=None, *, accumulate=False,
                          stream=None):
    """dx [R, D], dweight and dbias (or None) [D] (fp32, written or added to) of
    forge_layer_norm's output gradient dy [R, D], from its x, mean and rstd; dx
    may be dy or x itself."""
    gp, ldg, R, D = _rows(dy, "dy")
    xp, ldx, *in_ = _rows(x, "x")
    op, ldo, *out = _rows(dx, "dx")
    if in_ != [R, D] or out != [R, D]:
        raise ValueError(f"x and dx must be [R={R}, D={D}]")
    s = lib().forge_layer_norm_grad(gp, _float_code(dy), ldg, xp, _float_code(x), ldx,
                                    _vector(weight, D, "weight"), _vector(mean, R, "mean"),
                                    _vector(rstd, R, "rstd"), R, D, op, _float_code(dx), ldo,
                                    _vector(dweight, D, "dweight"), _vector(dbias, D, "dbias"),
                                    int(bool(accumulate)), _stream(stream, dy))
    _check(s, "forge_layer_norm_grad")


def _ints(t, n, what):
    """Pointer of an int32 tensor of n elements, or None."""
    if t is None:
        return None
    if (_codes or _all_codes()).get(t.dtype) == FORGE_I32 and t.numel() == n and t.is_cuda and \
            t.is_contiguous():
        return t.data_ptr()
    if t.numel() != n or _id_code(t) != FORGE_I32:
        raise ValueError(f"{what} must be int32 with {n} elements")
    return _ptr(t)


def forge_moe_route(logits, experts, weights, counts, offsets, *, slots=None, rows=None, live=None,
                    loss=None, normalize=True, stream=None):
    """The k experts of each token of logits [T, E] (bf16 or fp32, rows of any
    stride): experts (int32) and weights (fp32) [T, k], counts [E] and offsets
    [E + 1] (int32); where given the choices' packed rows slots [T, k], each
    packed row's token rows [T * k], the number of tokens that count live [1]
    (int32) and the balance loss [1] (fp32)."""
    lp, ld, T, E = _rows(logits, "logits")
    k = experts.shape[-1]
    if tuple(experts.shape) != (T, k) or tuple(weights.shape) != (T, k):
        raise ValueError(f"experts and weights must be [T={T}, k]")
    s = lib().forge_moe_route(lp, _float_code(logits), T, E, ld, k, int(bool(normalize)),
                              _ints(experts, T * k, "experts"), _vector(weights, T * k, "weights"),
                              _ints(counts, E, "counts"), _ints(offsets, E + 1, "offsets"),
                              _ints(_laid_out(slots, (T, k), "slots"), T * k, "slots"),
                              _ints(rows, T * k, "rows"),
                              _ints(live, 1, "live"), _vector(loss, 1, "loss"),
                              _stream(stream, logits))
    _check(s, "forge_moe_route")


def forge_moe_route_grad(logits, experts, counts, live, dlogits, *, grad_weights=None,
                         grad_loss=None, normalize=True, stream=None):
    """dlogits [T, E] (bf16 or fp32, rows of any stride; may be logits itself) of
    sum(grad_weights * weights) + grad_loss * loss, from what forge_moe_route
    gave."""
    lp, ld, T, E = _rows(logits, "logits")
    dp, ldo, *out = _rows(dlogits, "dlogits")
    k = experts.shape[-1]
    if out != [T, E] or tuple(experts.shape) != (T, k):
        raise ValueError(f"dlogits must be [T={T}, E={E}] and experts [T, k]")
    s = lib().forge_moe_route_grad(lp, _float_code(logits), T, E, ld, k, int(bool(normalize)),
                                   _ints(experts, T * k, "experts"), _ints(counts, E, "counts"),
                                   _ints(live, 1, "live"),
                                   _vector(_laid_out(grad_weights, (T, k), "grad_weights"), T * k,
                                           "grad_weights"),
                                   _vector(grad_loss, 1, "grad_loss"), dp, _float_code(dlogits),
                                   ldo, _stream(stream, logits))
    _check(s, "forge_moe_route_grad")


def _blocks(n):
    return -(-n // 128)


def _laid_out(t, shape, what):
    """t itself (or None), refused where its entries lie in another order than `shape`'s:
    [b, a] has as many as [a, b].  One dimension leaves the order to the caller."""
    if t is not None and t.dim() != 1 and t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    return t


def _byte_codes(t, what):
    """Pointer of a contiguous tensor of e4m3 codes (float8_e4m3fn, or uint8)."""
    import torch
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"{what} must be float8_e4m3fn or uint8, got {t.dtype}")
    return _ptr(t)


def forge_quantize_e4m3_blocks(x, codes, scales, *, block_rows=1, stream=None):
    """codes (float8_e4m3fn or uint8, x's shape) and scales (fp32) of x [R, C] or
    [E, R, C] (fp32 or bf16; rows of any stride in the 2-D form), a scale for each
    128 entries of a row (block_rows=1) or each square of 128 x 128 (128): [...,
    ceil(R / block_rows), ceil(C / 128)]."""
    if x.dim() == 3:
        E, R, C = x.shape
        xp, ldx = _ptr(x), C
    else:
        xp, ldx, R, C = _rows(x, "x")
        E = 1
    if tuple(codes.shape) != tuple(x.shape):
        raise ValueError("codes must have x's shape")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    down, across = -(-R // block_rows), _blocks(C)
    _laid_out(scales, (E, down, across) if x.dim() == 3 else (down, across), "scales")
    s = lib().forge_quantize_e4m3_blocks(xp, _float_code(x), ldx, E, R, C, block_rows,
                                         _byte_codes(codes, "codes"),
                                         _vector(scales, E * down * across, "scales"),
                                         _stream(stream, x))
    _check(s, "forge_quantize_e4m3_blocks")


def _linear_sizes(A, sA, W, sW, Y, transpose):
    """Pointers of the operands and (T, N, M), for W [N, M] or [E, N, M]."""
    *E, N, M = W.shape
    K, O = (M, N) if transpose else (N, M)
    T = A.shape[0]
    if tuple(A.shape) != (T, K) or tuple(Y.shape) != (T, O):
        raise ValueError(f"A [T, {K}] and Y [T, {O}] expected, got {tuple(A.shape)}, {tuple(Y.shape)}")
    of_A, of_W = (T, _blocks(K)), (*E, _blocks(N), _blocks(M))
    return (_byte_codes(A, "A"), _vector(_laid_out(sA, of_A, "sA"), math.prod(of_A), "sA"),
            _byte_codes(W, "W"), _vector(_laid_out(sW, of_W, "sW"), math.prod(of_W), "sW")), (T, N, M)


def forge_linear_e4m3(A, sA, W, sW, Y, *, transpose=False, stream=None):
    """Y [T, M] (bf16 or fp32) = A [T, N] times W [N, M], or with transpose Y [T, N]
    = A [T, M] times W transposed, of e4m3 codes: sA holds a scale for each 128
    entries of A's rows, sW for each 128 x 128 square of W (see
    forge_quantize_e4m3_blocks)."""
    if W.dim() != 2:
        raise ValueError("W must be [N, M]")
    ptrs, sizes = _linear_sizes(A, sA, W, sW, Y, transpose)
    s = lib().forge_linear_e4m3(*ptrs, _ptr(Y), _float_code(Y), *sizes, int(bool(transpose)),
                                _stream(stream, Y))
    _check(s, "forge_linear_e4m3")


def forge_grouped_linear_e4m3(A, sA, W, sW, offsets, Y, *, transpose=False, stream=None):
    """forge_linear_e4m3 by experts: W [E, N, M], sW [E, ...], and expert e's rows of A
    and Y are offsets[e] to offsets[e + 1] (int32 [E + 1] on the device); rows
    of no expert stay as they are in Y."""
    if W.dim() != 3:
        raise ValueError("W must be [E, N, M]")
    ptrs, sizes = _linear_sizes(A, sA, W, sW, Y, transpose)
    E = W.shape[0]
    s = lib().forge_grouped_linear_e4m3(*ptrs, _ints(offsets, E + 1, "offsets"), E, _ptr(Y),
                                        _float_code(Y), *sizes, int(bool(transpose)),
                                        _stream(stream, Y))
    _check(s, "forge_grouped_linear_e4m3")


def forge_status_string(status: int) -> str:
    return lib().forge_status_string(int(status)).decode()


def forge_get_device_status() -> int:
    return int(lib().forge_get_device_status())


def forge_selftest_wait_timeout(timeout_us: int, stream=None):
    import torch
    st = stream if stream is not None else torch.cuda.current_stream()
    _check(lib().forge_selftest_wait_timeout(int(timeout_us), ctypes.c_void_p(st.cuda_stream)),
           "forge_selftest_wait_timeout")


def forge_version() -> int:
    return int(lib().forge_version())
