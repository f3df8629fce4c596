"""FP8 block-scaled linear-layer kernels for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI of ``libfp8bs.so`` (``include/fp8bs.h``).
It only marshals arguments: tensors are allocated with torch on the current
CUDA device and every computation runs in the library's CUDA kernels on
torch's current stream.  There is no CPU fallback; if the library is missing
or cannot load, every call raises.

Calls keep the names and defaults of the DeepSeek-V3 inference kernels that
the pages describe:

* ``act_quant(x, block_size=128, scale_fmt=None) -> (q, s)``
* ``weight_dequant(x, s, block_size=128) -> y``
* ``fp8_gemm(a, a_s, b, b_s) -> y``
* ``fp8_linear(x, weight, weight_scale, scale_fmt=None) -> y``
* ``fp8_gemm_grouped(a, a_s, w, w_s, m_offsets) -> y``
* ``fp8_gemm_quant(a, a_s, b, b_s, out_scale_fmt=None) -> (q, s)`` (FP8 output)
* ``weight_quant(w, block_size=128, scale_fmt=None) -> (q, s)``

Around them stand the operators of the feed-forward block: the gated
projections (``fp8_gemm_gated``, ``fp8_gemm_gated_quant``,
``fp8_gemm_grouped_gated``, the whole block ``fp8_gated_ffn``), the gate's
backward pass (``gated_backward``, ``gated_backward_quant``), the linear layers on
4-bit weights (``weight_quant_int4``, ``weight_dequant_int4``, ``int4_linear``,
``int4_linear_gated``) and the norm and clipping of gradients (``grad_norm``,
``clip_grads``).
"""
import array
import ctypes
import functools
import os
import re

import torch

__all__ = [
    "act_quant", "act_quant_static", "act_dequant", "static_dequant",
    "weight_dequant", "weight_quant", "fp8_gemm", "fp8_linear", "fp8_linear_fused",
    "fp8_gemm_grouped", "fp8_gemm_quant", "fp8_gemm_rowwise", "act_quant_transposed",
    "fp8_transpose", "fp8_gemm_gated", "fp8_gemm_gated_quant", "fp8_gemm_grouped_gated",
    "fp8_gated_ffn", "gated_backward", "gated_backward_quant", "weight_quant_int4",
    "weight_dequant_int4", "int4_linear", "int4_linear_gated", "grad_norm", "clip_grads",
    "gemm_workspace_size", "gemm_plan", "linear_plan", "device_error", "lib",
    "Fp8bsError",
    "LIB_PATH", "HEADER_PATH",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8bs.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp8bs.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_SCALE = range(7)
DTYPE_BF16, DTYPE_F32 = 0, 1
SCALE_FMT_NONE, SCALE_FMT_UE8M0 = 0, 1


class Fp8bsError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (_STATUS_NAMES.get(status, status), message))
        self.status = status


_STATUS_NAMES = {OK: "FP8BS_OK", ERR_INVALID_ARG: "FP8BS_ERR_INVALID_ARG",
                 ERR_UNSUPPORTED: "FP8BS_ERR_UNSUPPORTED", ERR_WORKSPACE: "FP8BS_ERR_WORKSPACE",
                 ERR_CUDA: "FP8BS_ERR_CUDA", ERR_TIMEOUT: "FP8BS_ERR_TIMEOUT",
                 ERR_SCALE: "FP8BS_ERR_SCALE"}

_lib = None


def lib():
    """The loaded ``libfp8bs.so`` (ctypes.CDLL) with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libfp8bs.so is not built (python -m fp8_block_scaled_10_b200.build)")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "fp8bs_version": (i32, []),
        "fp8bs_status_string": (ctypes.c_char_p, [i32]),
        "fp8bs_last_error_message": (ctypes.c_char_p, []),
        "fp8bs_get_device_error": (i32, [p, ctypes.POINTER(i32)]),
        "fp8bs_act_quant": (i32, [p, i32, i64, i64, i64, i32, p, p, p]),
        "fp8bs_weight_dequant": (i32, [p, p, i64, i64, i64, p, i32, p]),
        "fp8bs_weight_quant": (i32, [p, i32, i64, i64, i64, i32, p, p, p]),
        "fp8bs_act_quant_static": (i32, [p, i32, i64, i64, i64, p, i64, p, p, p]),
        "fp8bs_act_quant_transposed": (i32, [p, i32, i64, i64, i64, i32, p, p, p]),
        "fp8bs_fp8_transpose": (i32, [p, p, i64, i64, i64, p, p, p]),
        "fp8bs_fp8_gemm_rowwise": (i32, [p, p, p, p, i64, i64, i64, i32, p, i32, p, sz, p]),
        "fp8bs_gemm_rowwise_workspace_size": (sz, [i64, i64, i64]),
        "fp8bs_act_dequant": (i32, [p, p, i64, i64, i64, i64, p, i32, p]),
        "fp8bs_gemm_workspace_size": (sz, [i64, i64, i64]),
        "fp8bs_gemm_plan_string": (ctypes.c_char_p, [i64, i64, i64]),
        "fp8bs_selftest_quotient": (i32, [p, p, p, i64, p]),
        "fp8bs_selftest_block_scale": (i32, [p, p, i64, i32, p]),
        "fp8bs_selftest_gemm_stall": (i32, [p, p, p, p, i64, i64, i64, p, p, sz, i32, p]),
        "fp8bs_fp8_gemm": (i32, [p, p, p, p, i64, i64, i64, p, p, sz, p]),
        "fp8bs_fp8_gemm_static_scratch": (i32, [p, p, p, p, i64, i64, i64, p, p]),
        "fp8bs_fp8_linear": (i32, [p, i64, i64, i32, p, p, i64, p, p, p, p, sz, p]),
        "fp8bs_linear_workspace_size": (sz, [i64, i64, i64]),
        "fp8bs_fp8_linear_fused": (i32, [p, i64, i64, i32, p, p, i64, p, p, p, p, sz, p]),
        "fp8bs_linear_plan_string": (ctypes.c_char_p, [i64, i64, i64]),
        "fp8bs_fp8_gemm_ue8m0": (i32, [p, p, p, p, i64, i64, i64, p, p, sz, p]),
        "fp8bs_fp8_gemm_f32": (i32, [p, p, p, p, i64, i64, i64, i32, p, p, sz, p]),
        "fp8bs_fp8_linear_ue8m0": (i32, [p, i64, i64, p, p, i64, p, p, p, p, sz, p]),
        "fp8bs_fp8_gemm_grouped_ue8m0": (i32, [i64, p, i64, p, p, p, p, i64, i64, p, p]),
        "fp8bs_fp8_gemm_grouped": (i32, [i64, p, i64, p, p, p, p, i64, i64, p, p]),
        "fp8bs_fp8_gemm_quant": (i32, [p, p, p, p, i64, i64, i64, i32, p, p, p, p]),
        "fp8bs_gemm_gated_workspace_size": (sz, [i64, i64, i64]),
        "fp8bs_fp8_gemm_gated": (i32, [p, p, p, p, p, p, i64, i64, i64, p, p, p, sz, p]),
        "fp8bs_fp8_gemm_gated_quant": (i32, [p, p, p, p, p, p, i64, i64, i64, i32, p, p, p, p, sz, p]),
        "fp8bs_fp8_gemm_grouped_gated": (i32, [i64, p, i64, p, p, p, p, p, p, i64, i64, p, p]),
        "fp8bs_gated_ffn_workspace_size": (sz, [i64, i64, i64, i64]),
        "fp8bs_fp8_gated_ffn": (i32, [p, i64, i64, p, i64, i32, p, p, p, p, i64, p, p, i64, p, p,
                                      sz, p]),
        "fp8bs_gated_backward": (i32, [p, p, i64, i64, p, p, p]),
        "fp8bs_gated_backward_quant": (i32, [p, p, i64, i64, i32, p, p, p, p, p, p, p]),
        "fp8bs_weight_quant_int4": (i32, [p, i32, i64, i64, i64, p, p, p]),
        "fp8bs_weight_dequant_int4": (i32, [p, p, i64, i64, i64, p, i32, p]),
        "fp8bs_int4_linear": (i32, [p, i64, p, p, i64, i64, i64, p, i32, p]),
        "fp8bs_int4_linear_gated": (i32, [p, i64, p, p, p, p, i64, i64, i64, p, i32, p]),
        "fp8bs_grad_norm_workspace_size": (sz, [i64]),
        "fp8bs_grad_norm": (i32, [p, p, p, i64, p, p, sz, p]),
        "fp8bs_clip_grads": (i32, [p, p, p, p, p, i64, p, p, p, sz, p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def header_symbols():
    """Names of the entry points that include/fp8bs.h declares."""
    text = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"FP8BS_API[^;(]*?\b(fp8bs_\w+)\s*\(", text)))


def _check(status):
    if status != OK:
        msg = lib().fp8bs_last_error_message().decode(errors="replace")
        raise Fp8bsError(status, msg)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(device):
    """The current stream's handle (the raw query: making a torch.cuda.Stream
    object for it takes 2 us)."""
    if device is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("fp8bs runs on CUDA tensors only (got a %s tensor)" % t.device)
        if not t.is_contiguous():
            raise ValueError("fp8bs expects contiguous tensors")
        if t.device != ts[0].device:
            raise ValueError("all operands must be on one device (%s and %s)"
                             % (ts[0].device, t.device))


def _here(*ts):
    """_need_cuda, first by the cheapest questions that answer it."""
    dev = ts[0].get_device()
    for t in ts:
        if t.get_device() != dev or dev < 0 or not t.is_contiguous():
            _need_cuda(*ts)


def _codes(t):
    """t, checked to hold e4m3fn codes (as float8_e4m3fn or uint8); the calls take
    its address alone."""
    if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
        raise TypeError("expected float8_e4m3fn or uint8 codes, got %s" % t.dtype)
    return t


def _scale_fmt(scale_fmt):
    if scale_fmt is None:
        return SCALE_FMT_NONE
    if scale_fmt == "ue8m0":
        return SCALE_FMT_UE8M0
    raise ValueError("scale_fmt must be None or 'ue8m0'")


def _io_dtype(dtype, what):
    """DTYPE_BF16 / DTYPE_F32 for a bfloat16 / float32 tensor dtype."""
    if dtype == torch.bfloat16:
        return DTYPE_BF16
    if dtype == torch.float32:
        return DTYPE_F32
    raise TypeError("%s must be torch.bfloat16 or torch.float32, got %s" % (what, dtype))


def _cdiv(a, b):
    return -(-a // b)


def _scales_like(s, shape, what):
    """Raise unless s is a float32 tensor of exactly ``shape``: the kernels read
    scales through raw pointers, so a short table would be read past its end."""
    if s.dtype is not torch.float32:
        raise TypeError("%s must be float32, got %s" % (what, s.dtype))
    if s.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(s.shape)))


def _gemm_operands(a, a_s, b, b_s):
    """Shape checks of fp8_gemm's operands -> (M, N, K)."""
    if b.dim() != 2:
        raise ValueError("b must be 2-D [N, K]")
    K = a.shape[-1]
    if b.shape[1] != K:
        raise ValueError("a [..., K] and b [N, K] disagree on K (%d vs %d)" % (K, b.shape[1]))
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    N = b.shape[0]
    _scales_like(a_s, (*a.shape[:-1], K // 128), "a_s")
    _scales_like(b_s, (_cdiv(N, 128), K // 128), "b_s")
    return a.numel() // K, N, K


def act_quant(x, block_size=128, scale_fmt=None):
    """Dynamic 1 x block_size quantization of the last dimension.

    Returns ``q`` (float8_e4m3fn, same shape as x) and ``s`` (float32,
    ``x.shape[:-1] + (x.shape[-1] // block_size,)``)."""
    _need_cuda(x)
    if x.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif x.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    if x.shape[-1] % block_size != 0:
        raise ValueError("last dimension must be a multiple of block_size")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty(*x.shape[:-1], cols // block_size, dtype=torch.float32, device=x.device)
    _check(lib().fp8bs_act_quant(_ptr(x), dt, rows, cols, block_size, _scale_fmt(scale_fmt),
                                 _ptr(q), _ptr(s), _stream(x.device)))
    return q, s


def _act_scales(s, lead, cols, block_size):
    """Row stride of a static scale vector [cols/block] (0) or a per-row table
    [..., cols/block] (cols/block)."""
    nblk = cols // block_size
    if s.dtype != torch.float32 or not s.is_contiguous():
        raise ValueError("scales must be contiguous float32")
    if tuple(s.shape) == (nblk,):
        return 0
    if tuple(s.shape) == tuple(lead) + (nblk,):
        return nblk
    raise ValueError("scales must be [cols/block] (static) or x.shape[:-1] + [cols/block]")


def act_quant_static(x, s, block_size=128, return_scales=False):
    """Static activation scheme: q = e4m3(x / s) with precomputed scales, no amax.

    s: float32 [cols/block_size] (one scale per block of channels, shared by
    every row) or a per-row table shaped like act_quant's.  Values beyond
    448 * s saturate.  With return_scales, also returns the per-row table
    ``x.shape[:-1] + (cols/block_size,)`` that fp8_gemm takes as a_s."""
    _need_cuda(x, s)
    if x.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif x.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError("x must be bfloat16 or float32")
    cols = x.shape[-1]
    if cols % block_size != 0:
        raise ValueError("last dimension must be a multiple of block_size")
    stride = _act_scales(s, x.shape[:-1], cols, block_size)
    rows = x.numel() // cols if cols else 0
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s_out = torch.empty(*x.shape[:-1], cols // block_size, dtype=torch.float32,
                        device=x.device) if return_scales else None
    _check(lib().fp8bs_act_quant_static(_ptr(x), dt, rows, cols, block_size, _ptr(s), stride,
                                        _ptr(q), _ptr(s_out), _stream(x.device)))
    return (q, s_out) if return_scales else q


def act_dequant(q, s, block_size=128, out_dtype=torch.float32):
    """y = q.float() * s per 1 x block_size block (the pages' static_dequant).

    s as for act_quant_static (a static vector or act_quant's per-row
    table); the fp32 product is returned as float32 or rounded to bfloat16."""
    q = _codes(q)
    _need_cuda(q, s)
    cols = q.shape[-1]
    if cols % block_size != 0:
        raise ValueError("last dimension must be a multiple of block_size")
    stride = _act_scales(s, q.shape[:-1], cols, block_size)
    rows = q.numel() // cols if cols else 0
    dt = _io_dtype(out_dtype, "out_dtype")
    y = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    _check(lib().fp8bs_act_dequant(_ptr(q), _ptr(s), stride, rows, cols, block_size, _ptr(y), dt,
                                   _stream(q.device)))
    return y


static_dequant = act_dequant


def weight_dequant(x, s, block_size=128, out_dtype=torch.bfloat16):
    """y[i, j] = x[i, j] * s[i // block_size, j // block_size] (fp32 product,
    rounded to ``out_dtype``, bfloat16 or float32)."""
    x = _codes(x)
    _need_cuda(x, s)
    if x.dim() != 2:
        raise ValueError("weight_dequant expects a 2-D weight")
    M, N = x.shape
    if tuple(s.shape) != (-(-M // block_size), -(-N // block_size)) or s.dtype != torch.float32:
        raise ValueError("s must be float32 of shape (cdiv(M, block), cdiv(N, block))")
    dt = _io_dtype(out_dtype, "out_dtype")
    y = torch.empty(M, N, dtype=out_dtype, device=x.device)
    _check(lib().fp8bs_weight_dequant(_ptr(x), _ptr(s), M, N, block_size, _ptr(y), dt,
                                      _stream(x.device)))
    return y


def weight_quant(w, block_size=128, scale_fmt=None):
    """block_size x block_size quantization of a dense 2-D weight -> (q e4m3fn, s float32)."""
    _need_cuda(w)
    if w.dim() != 2:
        raise ValueError("weight_quant expects a 2-D weight")
    dt = _io_dtype(w.dtype, "w")
    M, N = w.shape
    q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty(-(-M // block_size), -(-N // block_size), dtype=torch.float32, device=w.device)
    _check(lib().fp8bs_weight_quant(_ptr(w), dt, M, N, block_size, _scale_fmt(scale_fmt),
                                    _ptr(q), _ptr(s), _stream(w.device)))
    return q, s


def act_quant_transposed(x, block_size=128, scale_fmt=None):
    """Quantization in block_size x 1 column blocks, written transposed:
    act_quant(x.T) for a 2-D x [rows, cols] (rows % block_size == 0).

    Returns q [cols, rows] float8_e4m3fn and s [cols, rows // block_size]
    float32, the K-major operand of the weight-gradient GEMM."""
    _need_cuda(x)
    if x.dim() != 2:
        raise ValueError("act_quant_transposed expects a 2-D x")
    dt = _io_dtype(x.dtype, "x")
    rows, cols = x.shape
    q = torch.empty(cols, rows, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty(cols, rows // block_size, dtype=torch.float32, device=x.device)
    _check(lib().fp8bs_act_quant_transposed(_ptr(x), dt, rows, cols, block_size,
                                            _scale_fmt(scale_fmt), _ptr(q), _ptr(s),
                                            _stream(x.device)))
    return q, s


def fp8_transpose(q, s, block_size=128):
    """(q^T, s^T) of an FP8 matrix with block_size x block_size scales, exact."""
    q = _codes(q)
    _need_cuda(q, s)
    R, C = q.shape
    if tuple(s.shape) != (-(-R // block_size), -(-C // block_size)) or s.dtype != torch.float32:
        raise ValueError("s must be float32 of shape (cdiv(R, block), cdiv(C, block))")
    qt = torch.empty(C, R, dtype=torch.float8_e4m3fn, device=q.device)
    st = torch.empty(s.shape[1], s.shape[0], dtype=torch.float32, device=q.device)
    _check(lib().fp8bs_fp8_transpose(_ptr(q), _ptr(s.contiguous()), R, C, block_size,
                                     _ptr(qt), _ptr(st), _stream(q.device)))
    return qt, st


def fp8_gemm_rowwise(a, a_s, b, b_s, scale_fmt=None, out_dtype=torch.float32):
    """y = a @ b^T where both operands carry one scale per row and 128-wide
    K block (a_s [M, K/128], b_s [N, K/128]): the weight-gradient GEMM
    dW = dy^T x on act_quant_transposed(dy) and act_quant_transposed(x).
    out_dtype float32 (the default: weight gradients stay FP32) or bfloat16."""
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    a, b = _codes(a), _codes(b)
    if a.dim() != 2 or b.dim() != 2 or b.shape[1] != a.shape[1]:
        raise ValueError("a [M,K], a_s [M,K/128], b [N,K], b_s [N,K/128] expected")
    M, K = a.shape
    N = b.shape[0]
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    _scales_like(a_s, (M, K // 128), "a_s")
    _scales_like(b_s, (N, K // 128), "b_s")
    _need_cuda(a, a_s, b, b_s)
    y = torch.empty(M, N, dtype=out_dtype, device=a.device)
    nws = int(lib().fp8bs_gemm_rowwise_workspace_size(M, N, K))
    ws = torch.empty(nws, dtype=torch.uint8, device=a.device) if nws else None
    dt = DTYPE_F32 if out_dtype == torch.float32 else DTYPE_BF16
    _check(lib().fp8bs_fp8_gemm_rowwise(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), M, N, K,
                                        _scale_fmt(scale_fmt), _ptr(y), dt, _ptr(ws), nws,
                                        _stream(a.device)))
    return y


def gemm_workspace_size(M, N, K):
    """Bytes of scratch fp8_gemm needs for an M x N x K problem on this device."""
    return int(lib().fp8bs_gemm_workspace_size(M, N, K))


def linear_plan(M, N, K):
    """Which form fp8_linear takes for this shape on the current device
    (fused act_quant + GEMM in one launch, or the two launches)."""
    return lib().fp8bs_linear_plan_string(M, N, K).decode()


def gemm_plan(M, N, K):
    """The launch plan fp8_gemm uses for an M x N x K problem on this device."""
    return lib().fp8bs_gemm_plan_string(M, N, K).decode()


def _workspace(M, N, K, device):
    n = gemm_workspace_size(M, N, K)
    if n == 0:
        return None, 0
    return torch.empty(n, dtype=torch.uint8, device=device), n


def fp8_gemm(a, a_s, b, b_s, scale_fmt=None, out_dtype=torch.bfloat16):
    """y = a @ b^T on block-scaled FP8 operands.

    a: [..., K] e4m3fn, a_s: [..., K/128] float32, b: [N, K] e4m3fn,
    b_s: [cdiv(N,128), K/128] float32 -> y: [..., N] of out_dtype
    (torch.bfloat16, or torch.float32 for the unrounded FP32 accumulator).
    scale_fmt="ue8m0" promises that every scale is a power of two: the tensor
    core's block-scaled MMA applies them (at decode-sized M, up to 64 rows, the
    promotion kernel runs instead, with a check of the scales)."""
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    a, b = _codes(a), _codes(b)
    M, N, K = _gemm_operands(a, a_s, b, b_s)
    fmt = _scale_fmt(scale_fmt)
    _need_cuda(a, a_s, b, b_s)
    y = torch.empty(*a.shape[:-1], N, dtype=out_dtype, device=a.device)
    ws, nws = _workspace(M, N, K, a.device)
    if out_dtype == torch.float32:
        _check(lib().fp8bs_fp8_gemm_f32(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), M, N, K, fmt,
                                        _ptr(y), _ptr(ws), nws, _stream(a.device)))
        return y
    fn = lib().fp8bs_fp8_gemm_ue8m0 if fmt else lib().fp8bs_fp8_gemm
    _check(fn(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), M, N, K, _ptr(y), _ptr(ws), nws,
              _stream(a.device)))
    return y


def fp8_gemm_quant(a, a_s, b, b_s, out_scale_fmt=None, return_y=False):
    """fp8_gemm with an FP8 output: y = a @ b^T rounded to bf16, then quantized
    per 1x128 block of each row as act_quant(y, 128, out_scale_fmt) would.

    Returns (q e4m3fn [..., N], s float32 [..., N/128]), plus the bf16 y when
    return_y.  N must be a multiple of 128."""
    a, b = _codes(a), _codes(b)
    M, N, K = _gemm_operands(a, a_s, b, b_s)
    if N % 128 != 0:
        raise ValueError("N=%d must be a multiple of 128 for an FP8 output" % N)
    _need_cuda(a, a_s, b, b_s)
    q = torch.empty(*a.shape[:-1], N, dtype=torch.uint8, device=a.device)
    s = torch.empty(*a.shape[:-1], N // 128, dtype=torch.float32, device=a.device)
    y = torch.empty(*a.shape[:-1], N, dtype=torch.bfloat16, device=a.device) if return_y else None
    _check(lib().fp8bs_fp8_gemm_quant(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), M, N, K,
                                      _scale_fmt(out_scale_fmt), _ptr(q), _ptr(s), _ptr(y),
                                      _stream(a.device)))
    q = q.view(torch.float8_e4m3fn)
    return (q, s, y) if return_y else (q, s)


def fp8_linear(x, weight, weight_scale, scale_fmt=None, return_quant=False,
               weight_scale_fmt=None):
    """FP8 linear forward: act_quant(x) then fp8_gemm with the block-scaled weight.

    x: [..., K] bfloat16, weight: [N, K] e4m3fn, weight_scale: [cdiv(N,128), K/128].
    With scale_fmt="ue8m0" and weight_scale_fmt="ue8m0" (power-of-two weight
    scales) the GEMM is the ue8m0 entry (block-scaled MMA; promotion kernel at
    decode-sized M)."""
    w = _codes(weight)
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError("weight must be [N, K] with K = x.shape[-1]")
    K = x.shape[-1]
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    N = w.shape[0]
    _scales_like(weight_scale, (_cdiv(N, 128), K // 128), "weight_scale")
    _need_cuda(x, w, weight_scale)
    M = x.numel() // K
    y = torch.empty(*x.shape[:-1], N, dtype=torch.bfloat16, device=x.device)
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty(*x.shape[:-1], K // 128, dtype=torch.float32, device=x.device)
    if _scale_fmt(scale_fmt) and _scale_fmt(weight_scale_fmt):
        ws, nws = _workspace(M, N, K, x.device)
        _check(lib().fp8bs_fp8_linear_ue8m0(_ptr(x), M, K, _ptr(w), _ptr(weight_scale), N,
                                            _ptr(y), _ptr(q), _ptr(s), _ptr(ws), nws,
                                            _stream(x.device)))
    else:
        nws = int(lib().fp8bs_linear_workspace_size(M, N, K))
        ws = torch.empty(nws, dtype=torch.uint8, device=x.device) if nws else None
        _check(lib().fp8bs_fp8_linear(_ptr(x), M, K, _scale_fmt(scale_fmt), _ptr(w),
                                      _ptr(weight_scale), N, _ptr(y), _ptr(q), _ptr(s), _ptr(ws),
                                      nws, _stream(x.device)))
    return (y, q, s) if return_quant else y


def fp8_linear_fused(x, weight, weight_scale, scale_fmt=None, return_quant=False):
    """The FP8 linear forward as one launch: the SMs the GEMM's tiles leave
    idle quantize x (act_quant, bit-identical q and s) while the GEMM
    consumes it.  Raises (FP8BS_ERR_UNSUPPORTED) where no such launch exists:
    decode-sized M, or tiles that fill the GPU.  fp8_linear picks this form
    itself when the planner expects it to be faster (linear_plan names the
    choice).  x: [..., K] bfloat16, weight: [N, K] e4m3fn, weight_scale:
    [cdiv(N,128), K/128]; scale_fmt sets the activation scales' format."""
    w = _codes(weight)
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError("weight must be [N, K] with K = x.shape[-1]")
    K = x.shape[-1]
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    N = w.shape[0]
    _scales_like(weight_scale, (_cdiv(N, 128), K // 128), "weight_scale")
    _need_cuda(x, w, weight_scale)
    M = x.numel() // K
    y = torch.empty(*x.shape[:-1], N, dtype=torch.bfloat16, device=x.device)
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty(*x.shape[:-1], K // 128, dtype=torch.float32, device=x.device)
    nws = int(lib().fp8bs_linear_workspace_size(M, N, K))
    ws = torch.empty(nws, dtype=torch.uint8, device=x.device) if nws else None
    _check(lib().fp8bs_fp8_linear_fused(_ptr(x), M, K, _scale_fmt(scale_fmt), _ptr(w),
                                        _ptr(weight_scale), N, _ptr(y), _ptr(q), _ptr(s),
                                        _ptr(ws), nws, _stream(x.device)))
    return (y, q, s) if return_quant else y


def fp8_gemm_grouped(a, a_s, w, w_s, m_offsets, scale_fmt=None):
    """Per-expert FP8 GEMMs over rows grouped contiguously by expert.

    a: [M_total, K] e4m3fn, a_s: [M_total, K/128], w: [G, N, K] e4m3fn,
    w_s: [G, cdiv(N,128), K/128], m_offsets: [G+1] int64 on the device."""
    a, w = _codes(a), _codes(w)
    if m_offsets.dtype != torch.int64:
        raise TypeError("m_offsets must be int64")
    if a.dim() != 2 or w.dim() != 3 or w.shape[2] != a.shape[1]:
        raise ValueError("a [M_total, K] and w [G, N, K] expected")
    G, N, K = w.shape
    M = a.shape[0]
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    if tuple(m_offsets.shape) != (G + 1,):
        raise ValueError("m_offsets must have shape (G + 1,) = (%d,)" % (G + 1))
    _scales_like(a_s, (M, K // 128), "a_s")
    _scales_like(w_s, (G, _cdiv(N, 128), K // 128), "w_s")
    _need_cuda(a, a_s, w, w_s, m_offsets)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    fn = lib().fp8bs_fp8_gemm_grouped_ue8m0 if _scale_fmt(scale_fmt) else lib().fp8bs_fp8_gemm_grouped
    _check(fn(G, _ptr(m_offsets), M, _ptr(a), _ptr(a_s), _ptr(w), _ptr(w_s), N, K, _ptr(y),
              _stream(a.device)))
    return y


def _on_device(fn):
    """Runs an operator with its first tensor's device current: the library plans
    and launches on the current device.  (A call on the current device, the
    usual one, costs one comparison.)"""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        for t in args[:1] or kwargs.values():   # keywords come in any order
            if isinstance(t, (list, tuple)) and t:
                t = t[0]
            if getattr(t, "is_cuda", False):
                break
        else:
            return fn(*args, **kwargs)   # which refuses
        if t.get_device() == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(t.device):
            return fn(*args, **kwargs)
    return call


def _gated_operands(a, a_s, w_gate, w_gate_s, w_up, w_up_s):
    """Checks of the gated projections' operands -> (M, N, K)."""
    _codes(a), _codes(w_gate), _codes(w_up)
    if w_gate.shape != w_up.shape:
        raise ValueError("w_gate and w_up must have one shape, got %s and %s"
                         % (tuple(w_gate.shape), tuple(w_up.shape)))
    M, N, K = _gemm_operands(a, a_s, w_gate, w_gate_s)
    _scales_like(w_up_s, w_gate_s.shape, "w_up_s")
    if N == 0:
        raise ValueError("the weights have no rows")
    _here(a, a_s, w_gate, w_gate_s, w_up, w_up_s)
    return M, N, K


def _gated_workspace(M, N, K, device):
    n = int(lib().fp8bs_gemm_gated_workspace_size(M, N, K))
    return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n


@_on_device
def fp8_gemm_gated(a, a_s, w_gate, w_gate_s, w_up, w_up_s, return_gu=False):
    """h = silu(a @ w_gate^T) * (a @ w_up^T) on block-scaled FP8 operands, one
    kernel: the gated projections of a feed-forward block.

    a: [..., K] e4m3fn, a_s: [..., K/128] float32 (act_quant's output),
    w_gate, w_up: [N, K] e4m3fn, their scales [cdiv(N,128), K/128] float32 (any
    positive scales; powers of two take the same kernel, not the block-scaled MMA of
    fp8_gemm's scale_fmt="ue8m0") -> h: [..., N] bfloat16.  With
    return_gu also the bfloat16 pre-activations [..., 2N], gate first, which
    gated_backward takes."""
    M, N, K = _gated_operands(a, a_s, w_gate, w_gate_s, w_up, w_up_s)
    h = torch.empty(*a.shape[:-1], N, dtype=torch.bfloat16, device=a.device)
    gu = torch.empty(*a.shape[:-1], 2 * N, dtype=torch.bfloat16, device=a.device) if return_gu else None
    ws, nws = _gated_workspace(M, N, K, a.device)
    _check(lib().fp8bs_fp8_gemm_gated(_ptr(a), _ptr(a_s), _ptr(w_gate), _ptr(w_gate_s), _ptr(w_up),
                                      _ptr(w_up_s), M, N, K, _ptr(h), _ptr(gu), _ptr(ws), nws,
                                      _stream(a.device)))
    return (h, gu) if return_gu else h


@_on_device
def fp8_gemm_gated_quant(a, a_s, w_gate, w_gate_s, w_up, w_up_s, out_scale_fmt=None,
                         return_h=False):
    """fp8_gemm_gated with an FP8 output for the down projection: h rounded to
    bf16, then quantized as act_quant(h, 128, out_scale_fmt) would.

    Returns (q e4m3fn [..., N], s float32 [..., N/128]), plus h when return_h.
    N must be a multiple of 128."""
    fmt = _scale_fmt(out_scale_fmt)
    M, N, K = _gated_operands(a, a_s, w_gate, w_gate_s, w_up, w_up_s)
    if N % 128 != 0:
        raise ValueError("N=%d must be a multiple of 128 for an FP8 output" % N)
    q = torch.empty(*a.shape[:-1], N, dtype=torch.float8_e4m3fn, device=a.device)
    s = torch.empty(*a.shape[:-1], N // 128, dtype=torch.float32, device=a.device)
    h = torch.empty(*a.shape[:-1], N, dtype=torch.bfloat16, device=a.device) if return_h else None
    ws, nws = _gated_workspace(M, N, K, a.device)
    _check(lib().fp8bs_fp8_gemm_gated_quant(_ptr(a), _ptr(a_s), _ptr(w_gate), _ptr(w_gate_s),
                                            _ptr(w_up), _ptr(w_up_s), M, N, K, fmt, _ptr(q),
                                            _ptr(s), _ptr(h), _ptr(ws), nws, _stream(a.device)))
    return (q, s, h) if return_h else (q, s)


@_on_device
def fp8_gemm_grouped_gated(a, a_s, w_gate, w_gate_s, w_up, w_up_s, m_offsets):
    """fp8_gemm_gated per expert, over rows grouped contiguously by expert (h
    alone: the pre-activations that gated_backward takes come from two
    fp8_gemm_grouped calls).

    a: [M_total, K] e4m3fn, a_s: [M_total, K/128], w_gate, w_up: [G, N, K], their
    scales [G, cdiv(N,128), K/128], m_offsets: [G+1] int64 on the device ->
    h: [M_total, N] bfloat16 (rows that belong to no expert are not written)."""
    a, w_gate, w_up = _codes(a), _codes(w_gate), _codes(w_up)
    if m_offsets.dtype != torch.int64:
        raise TypeError("m_offsets must be int64")
    if a.dim() != 2 or w_gate.dim() != 3 or w_gate.shape[2] != a.shape[1]:
        raise ValueError("a [M_total, K] and w_gate, w_up [G, N, K] expected")
    if w_gate.shape != w_up.shape:
        raise ValueError("w_gate and w_up must have one shape, got %s and %s"
                         % (tuple(w_gate.shape), tuple(w_up.shape)))
    G, N, K = w_gate.shape
    M = a.shape[0]
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    if tuple(m_offsets.shape) != (G + 1,):
        raise ValueError("m_offsets must have shape (G + 1,) = (%d,)" % (G + 1))
    _scales_like(a_s, (M, K // 128), "a_s")
    _scales_like(w_gate_s, (G, _cdiv(N, 128), K // 128), "w_gate_s")
    _scales_like(w_up_s, (G, _cdiv(N, 128), K // 128), "w_up_s")
    _here(a, a_s, w_gate, w_gate_s, w_up, w_up_s, m_offsets)
    h = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    _check(lib().fp8bs_fp8_gemm_grouped_gated(G, _ptr(m_offsets), M, _ptr(a), _ptr(a_s),
                                              _ptr(w_gate), _ptr(w_gate_s), _ptr(w_up),
                                              _ptr(w_up_s), N, K, _ptr(h), _stream(a.device)))
    return h


@_on_device
def fp8_gated_ffn(x, w_gate, w_gate_s, w_up, w_up_s, w_down, w_down_s, scale_fmt=None,
                  x_scales=None):
    """The whole gated feed-forward block, forward: act_quant(x), the gated
    projections with an FP8 output, the down projection.

    x: [..., K] bfloat16, w_gate, w_up: [N, K], w_down: [K_out, N] e4m3fn with
    128 x 128 block scales; N a multiple of 128; scale_fmt is the format of both
    activations' scales -> y: [..., K_out] bfloat16.  x_scales: the scales of x
    where the caller has them (the static scheme: [K/128], or a per-row table
    x.shape[:-1] + [K/128], as act_quant_static takes)."""
    w_gate, w_up, w_down = _codes(w_gate), _codes(w_up), _codes(w_down)
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if w_gate.dim() != 2 or w_down.dim() != 2 or w_down.shape[1] != w_gate.shape[0]:
        raise ValueError("w_gate, w_up [N, K] and w_down [K_out, N] expected")
    N, K = w_gate.shape
    k_out = w_down.shape[0]
    if x.dim() == 0 or x.shape[-1] != K or K <= 0 or K % 128 != 0:
        raise ValueError("x [..., K] and w_gate [N, K] with K a multiple of 128 expected")
    if N <= 0 or N % 128 != 0:
        raise ValueError("N=%d must be a positive multiple of 128" % N)
    if w_up.shape != w_gate.shape:
        raise ValueError("w_gate and w_up must have one shape, got %s and %s"
                         % (tuple(w_gate.shape), tuple(w_up.shape)))
    _scales_like(w_gate_s, (N // 128, K // 128), "w_gate_s")
    _scales_like(w_up_s, (N // 128, K // 128), "w_up_s")
    _scales_like(w_down_s, (_cdiv(k_out, 128), N // 128), "w_down_s")
    stride = 0 if x_scales is None else _act_scales(x_scales, x.shape[:-1], K, 128)
    fmt = _scale_fmt(scale_fmt)
    _here(x, w_gate, w_gate_s, w_up, w_up_s, w_down, w_down_s,
               *(() if x_scales is None else (x_scales,)))
    M = x.numel() // K
    y = torch.empty(*x.shape[:-1], k_out, dtype=torch.bfloat16, device=x.device)
    nws = int(lib().fp8bs_gated_ffn_workspace_size(M, N, K, k_out))
    ws = torch.empty(nws, dtype=torch.uint8, device=x.device) if nws else None
    _check(lib().fp8bs_fp8_gated_ffn(_ptr(x), M, K, _ptr(x_scales), stride, fmt, _ptr(w_gate),
                                     _ptr(w_gate_s), _ptr(w_up), _ptr(w_up_s), N, _ptr(w_down),
                                     _ptr(w_down_s), k_out, _ptr(y), _ptr(ws), nws,
                                     _stream(x.device)))
    return y


def _gate_operands(gu, dh):
    """Checks of the gate's backward pass -> (M, N)."""
    if gu.dtype != torch.bfloat16 or dh.dtype != torch.bfloat16:
        raise TypeError("gu and dh must be bfloat16")
    N = dh.shape[-1]
    if tuple(gu.shape) != tuple(dh.shape[:-1]) + (2 * N,):
        raise ValueError("gu must be dh.shape[:-1] + (2 N,), got %s and %s"
                         % (tuple(gu.shape), tuple(dh.shape)))
    _here(gu, dh)
    return (dh.numel() // N if N else 0), N


@_on_device
def gated_backward(gu, dh, return_h=False):
    """The backward pass of h = silu(g) * u: dgu from the pre-activations and dh.

    gu: [..., 2N] bfloat16 as fp8_gemm_gated returns it (gate first), dh: [..., N]
    bfloat16 -> dgu: [..., 2N] bfloat16; with return_h also h [..., N] again."""
    M, N = _gate_operands(gu, dh)
    dgu = torch.empty_like(gu)
    h = torch.empty_like(dh) if return_h else None
    _check(lib().fp8bs_gated_backward(_ptr(gu), _ptr(dh), M, N, _ptr(dgu), _ptr(h),
                                      _stream(gu.device)))
    return (dgu, h) if return_h else dgu


@_on_device
def gated_backward_quant(gu, dh, scale_fmt=None):
    """gated_backward with its results quantized for the FP8 gradient GEMMs, in
    one pass, by act_quant's rule from the fp32 values.

    gu: [M, 2N], dh: [M, N] bfloat16, N a multiple of 128.  Returns (with Mp = M
    rounded up to 128, codes e4m3fn, scales float32)

    * q [M, 2N], s [M, 2N/128]: dgu, the operand of dx;
    * qt [2N, Mp], st [2N, Mp/128]: dgu transposed, the operand of dW_gate, dW_up;
    * ht [N, Mp], hts [N, Mp/128]: h transposed, the operand of dW_down.

    Codes of the tokens past M are zero: fp8_gemm_rowwise over Mp tokens sums over
    M (act_quant_transposed of an operand padded with zero rows fits them)."""
    fmt = _scale_fmt(scale_fmt)
    if dh.dim() != 2:
        raise ValueError("gu [M, 2N] and dh [M, N] expected")
    if dh.shape[1] % 128 != 0 or dh.shape[1] == 0:
        raise ValueError("N=%d must be a positive multiple of 128" % dh.shape[1])
    M, N = _gate_operands(gu, dh)
    mp, dev = _cdiv(M, 128) * 128, gu.device
    q = torch.empty(M, 2 * N, dtype=torch.float8_e4m3fn, device=dev)
    s = torch.empty(M, 2 * N // 128, dtype=torch.float32, device=dev)
    qt = torch.empty(2 * N, mp, dtype=torch.float8_e4m3fn, device=dev)
    st = torch.empty(2 * N, mp // 128, dtype=torch.float32, device=dev)
    ht = torch.empty(N, mp, dtype=torch.float8_e4m3fn, device=dev)
    hts = torch.empty(N, mp // 128, dtype=torch.float32, device=dev)
    _check(lib().fp8bs_gated_backward_quant(_ptr(gu), _ptr(dh), M, N, fmt, _ptr(q), _ptr(s),
                                            _ptr(qt), _ptr(st), _ptr(ht), _ptr(hts), _stream(dev)))
    return q, s, qt, st, ht, hts


@_on_device
def weight_quant_int4(w, group_size=128):
    """4-bit quantization of a dense weight in groups of group_size (32, 64 or
    128) input channels: w [N, K] bfloat16 or float32, K a multiple of 128 ->
    q uint8 [N, K/2] (packed, layout in include/fp8bs.h), s float32 [N, K/group_size]."""
    if w.dim() != 2:
        raise ValueError("weight_quant_int4 expects a 2-D weight")
    dt = _io_dtype(w.dtype, "w")
    N, K = w.shape
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    if group_size not in (32, 64, 128):
        raise ValueError("group_size must be 32, 64 or 128")
    _here(w)
    q = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
    s = torch.empty(N, K // group_size, dtype=torch.float32, device=w.device)
    _check(lib().fp8bs_weight_quant_int4(_ptr(w), dt, N, K, group_size, _ptr(q), _ptr(s),
                                         _stream(w.device)))
    return q, s


def _int4_operands(q, s, what):
    """Checks of a packed 4-bit weight -> (N, K, group size)."""
    if q.dtype != torch.uint8 or q.dim() != 2:
        raise ValueError("%s must be packed uint8 codes [N, K/2]" % what)
    N, K = q.shape
    K *= 2
    if K <= 0 or K % 128 != 0:
        raise ValueError("K=%d must be a positive multiple of 128" % K)
    group = K // s.shape[1] if s.dim() == 2 and s.shape[1] else 0
    if group not in (32, 64, 128) or tuple(s.shape) != (N, K // group):
        raise ValueError("%s's scales must be [N, K/group] with a group of 32, 64 or 128, got %s"
                         % (what, tuple(s.shape)))
    if s.dtype != torch.float32:
        raise TypeError("%s's scales must be float32, got %s" % (what, s.dtype))
    return N, K, group


@_on_device
def weight_dequant_int4(q, s, out_dtype=torch.bfloat16):
    """y [N, K] = (code - 8) * s per group of a packed 4-bit weight (fp32 product,
    rounded to ``out_dtype``, bfloat16 or float32)."""
    N, K, group = _int4_operands(q, s, "q")
    dt = _io_dtype(out_dtype, "out_dtype")
    _here(q, s)
    y = torch.empty(N, K, dtype=out_dtype, device=q.device)
    _check(lib().fp8bs_weight_dequant_int4(_ptr(q), _ptr(s), N, K, group, _ptr(y), dt,
                                           _stream(q.device)))
    return y


def _int4_tokens(x, K, out_dtype):
    if x.dtype is not torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if x.dim() == 0 or x.shape[-1] != K:
        raise ValueError("x [..., K] and the weight disagree on K (%s vs %d)" % (tuple(x.shape), K))
    return x.numel() // K, _io_dtype(out_dtype, "out_dtype")


@_on_device
def int4_linear(x, q, s, out_dtype=torch.bfloat16):
    """y = x @ W^T on a packed 4-bit weight, for decode-sized token counts: the
    weight is read and expanded once per 32 tokens, so that from about 128 tokens on
    weight_dequant_int4 and a bf16 product take less time.

    x: [..., K] bfloat16, q: uint8 [N, K/2], s: float32 [N, K/group] (as
    weight_quant_int4 returns them) -> y: [..., N] bfloat16 or float32."""
    N, K, group = _int4_operands(q, s, "q")
    M, dt = _int4_tokens(x, K, out_dtype)
    _here(x, q, s)
    y = torch.empty(*x.shape[:-1], N, dtype=out_dtype, device=x.device)
    _check(lib().fp8bs_int4_linear(_ptr(x), M, _ptr(q), _ptr(s), N, K, group, _ptr(y), dt,
                                   _stream(x.device)))
    return y


@_on_device
def int4_linear_gated(x, q_gate, s_gate, q_up, s_up, out_dtype=torch.bfloat16):
    """h = silu(x @ Wg^T) * (x @ Wu^T) on two packed 4-bit weights of one shape
    and group size, one kernel; arguments as for int4_linear."""
    N, K, group = _int4_operands(q_gate, s_gate, "q_gate")
    if _int4_operands(q_up, s_up, "q_up") != (N, K, group):
        raise ValueError("q_gate and q_up must have one shape and group size")
    M, dt = _int4_tokens(x, K, out_dtype)
    _here(x, q_gate, s_gate, q_up, s_up)
    h = torch.empty(*x.shape[:-1], N, dtype=out_dtype, device=x.device)
    _check(lib().fp8bs_int4_linear_gated(_ptr(x), M, _ptr(q_gate), _ptr(s_gate), _ptr(q_up),
                                         _ptr(s_up), N, K, group, _ptr(h), dt, _stream(x.device)))
    return h


_GRAD_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _grad_arrays(grads, what):
    """(pointers, types) of a list of gradient tensors, as C arrays."""
    if not isinstance(grads, (list, tuple)) or not grads:
        raise ValueError("%s must be a list of tensors, one at least" % what)
    try:
        types = array.array("i", [_GRAD_DTYPES[g.dtype] for g in grads])
    except (KeyError, AttributeError):
        raise TypeError("%s must be bfloat16 or float32 tensors" % what) from None
    devices = set(map(torch.Tensor.get_device, grads))
    if len(devices) > 1 or -1 in devices or not all(map(torch.Tensor.is_contiguous, grads)):
        _need_cuda(*grads)   # which says what is wrong
    return array.array("Q", map(torch.Tensor.data_ptr, grads)), types


def _sizes(grads):
    return array.array("q", map(torch.Tensor.numel, grads))


def _address(a):
    return a.buffer_info()[0]


def _norm_buffers(n, device):
    nws = int(lib().fp8bs_grad_norm_workspace_size(n))
    return (torch.empty((), dtype=torch.float32, device=device),
            torch.empty(nws, dtype=torch.uint8, device=device), nws)


@_on_device
def grad_norm(grads):
    """The global 2-norm over a list of gradient tensors (bfloat16 or float32,
    contiguous, one device), accumulated in 64 bits: a 0-dim float32 tensor."""
    ptrs, types = _grad_arrays(grads, "grads")
    n, dev = len(grads), grads[0].device
    sizes = _sizes(grads)
    norm, ws, nws = _norm_buffers(n, dev)
    _check(lib().fp8bs_grad_norm(_address(ptrs), _address(sizes), _address(types), n, _ptr(norm),
                                 _ptr(ws), nws, _stream(dev)))
    return norm


@_on_device
def clip_grads(grads, max_norm, out=None):
    """Scales a list of gradients by min(1, max_norm / (norm + 1e-6)), with norm
    their global 2-norm.  Returns (out, norm): norm is the 0-dim float32 norm
    before clipping.

    out: None (in place; nothing is written when nothing is clipped) or a list of
    bfloat16 or float32 tensors of the gradients' shapes that receive the
    scaled values.  Outputs may not overlap one another nor another tensor's
    gradient.  A NaN norm makes every output NaN, an infinite one scales by 0 (with
    max_norm=inf too)."""
    ptrs, types = _grad_arrays(grads, "grads")
    n, dev = len(grads), grads[0].device
    if out is None:
        out, out_ptrs, out_types = grads, ptrs, types
    else:
        out_ptrs, out_types = _grad_arrays(out, "out")
        if len(out) != n or any([o.shape != g.shape for o, g in zip(out, grads)]):
            raise ValueError("out must have the gradients' shapes")
        if out[0].get_device() != grads[0].get_device():
            raise ValueError("out and grads must be on one device")
    sizes = _sizes(grads)
    norm, ws, nws = _norm_buffers(n, dev)
    _check(lib().fp8bs_clip_grads(_address(ptrs), _address(out_ptrs), _address(sizes), _address(types),
                                  _address(out_types), n, ctypes.byref(ctypes.c_double(max_norm)),
                                  _ptr(norm), _ptr(ws), nws, _stream(dev)))
    return out, norm


def device_error(device=None):
    """Synchronize the current stream, then read and clear the device error word."""
    code = ctypes.c_int(0)
    device = torch.device(device) if device is not None else None
    _check(lib().fp8bs_get_device_error(_stream(device), ctypes.byref(code)))
    return code.value
