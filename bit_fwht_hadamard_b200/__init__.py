"""libqfp4: B200-native FP4 microscaling quantization and block-scaled FP4 GEMM.

Thin Python binding over the C ABI in ``include/qfp4.h``.  Every step of the
method runs in the CUDA kernels of ``libqfp4.so``; this module only marshals
arguments (torch tensors for device memory, CUDA streams) and allocates the
output tensors.  There is no CPU fallback: if the library is missing the
import of the functions below raises.

The ``qfp4_*`` functions mirror the C entry points one to one (pointers as
integers); ``quantize``, ``quantize_mxfp8``, ``dequantize``, ``gemm``,
``gemm_fused_rq``, ``gemm_epilogue``, ``linear_forward_epilogue``,
``epilogue_backward``, ``dropout``, ``layernorm_forward`` and
``layernorm_backward`` are conveniences that allocate outputs.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import c_int, c_int64, c_size_t, c_uint64, c_void_p, c_char_p, c_double, c_float

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqfp4.so")

MXFP4, NVFP4, MXFP8 = 0, 1, 2
RNE, SR = 0, 1
BF16, F32 = 0, 1
GRAN_TENSOR, GRAN_ROW, GRAN_GROUP16, GRAN_GROUP32 = 0, 1, 2, 3
SCALE_DEFAULT, SCALE_OCP_FLOOR, SCALE_E4M3_UP = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
OK, ERR_ARG, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_CUDA, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6
DEV_ERR_TIMEOUT = 1

EXPORTS = [
    "qfp4_quantize_workspace_bytes", "qfp4_quantize", "qfp4_quantize_ex", "qfp4_quantize_mxfp8", "qfp4_quantize_fp32scale",
    "qfp4_dequantize", "qfp4_gemm_workspace_bytes", "qfp4_gemm_blockscaled", "qfp4_gemm_fused_rq_workspace_bytes",
    "qfp4_gemm_fused_rq", "qfp4_gemm_fused_rq_ex", "qfp4_gemm_fused_rq_workspace_layout", "qfp4_gemm_blockscaled_noalloc",
    "qfp4_linear_forward_workspace_bytes", "qfp4_linear_forward", "qfp4_linear_backward_workspace_bytes",
    "qfp4_linear_backward", "qfp4_gemm_epilogue_workspace_bytes", "qfp4_gemm_epilogue",
    "qfp4_linear_forward_epilogue", "qfp4_epilogue_backward_workspace_bytes", "qfp4_epilogue_backward",
    "qfp4_dropout", "qfp4_layernorm_forward", "qfp4_layernorm_backward_workspace_bytes", "qfp4_layernorm_backward",
    "qfp4_kl_calibrate_workspace_bytes", "qfp4_kl_calibrate",
    "qfp4_status_string", "qfp4_last_device_error", "qfp4_selftest_wait_timeout", "qfp4_version",
    "qfp4_launch_count",
]

_lib = None


class Epilogue(ctypes.Structure):
    """The C struct qfp4_epilogue (pointers as integers, or None)."""
    _fields_ = [("bias", c_void_p), ("residual", c_void_p), ("preact", c_void_p), ("step", c_void_p),
                ("seed", c_uint64), ("dropout_p", c_double), ("bias_dt", c_int), ("residual_dt", c_int),
                ("act", c_int)]


class QFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({status_string(status)})")
        self.status = status


def lib():
    """Load libqfp4.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libqfp4.so not built at {LIB_PATH}; run __graft_entry__.build() or "
                              f"python -m bit_fwht_hadamard_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        P = c_void_p
        L.qfp4_quantize_workspace_bytes.restype = c_size_t
        L.qfp4_quantize_workspace_bytes.argtypes = [c_int64, c_int64, c_int, c_int, c_int]
        L.qfp4_quantize.restype = c_int
        L.qfp4_quantize.argtypes = [P, c_int, c_int64, c_int64, c_int, c_int, c_int, c_int, c_int, c_uint64,
                                    P, P, P, P, P, P, c_size_t, P]
        L.qfp4_quantize_ex.restype = c_int
        L.qfp4_quantize_ex.argtypes = [P, c_int, c_int64, c_int64, c_int, c_int, c_int, c_int, c_int, c_int,
                                       c_uint64, P, P, P, P, P, P, P, P, c_size_t, P]
        L.qfp4_quantize_mxfp8.restype = c_int
        L.qfp4_quantize_mxfp8.argtypes = [P, c_int, c_int64, c_int64, c_int, c_uint64, P, P, P, P, P]
        L.qfp4_quantize_fp32scale.restype = c_int
        L.qfp4_quantize_fp32scale.argtypes = [P, c_int, c_int64, c_int64, c_int, P, P, P, c_size_t, P]
        L.qfp4_dequantize.restype = c_int
        L.qfp4_dequantize.argtypes = [P, P, P, c_int64, c_int64, c_int, c_int, P, P]
        L.qfp4_gemm_workspace_bytes.restype = c_size_t
        L.qfp4_gemm_workspace_bytes.argtypes = [c_int64, c_int64, c_int64, c_int]
        L.qfp4_gemm_blockscaled.restype = c_int
        L.qfp4_gemm_blockscaled.argtypes = [P, P, P, P, P, P, c_int64, c_int64, c_int64, c_int, c_int, P, P,
                                            c_size_t, P]
        L.qfp4_gemm_blockscaled_noalloc.restype = c_int
        L.qfp4_gemm_blockscaled_noalloc.argtypes = [P, P, P, P, P, P, c_int64, c_int64, c_int64, c_int, c_int, P, P]
        L.qfp4_gemm_fused_rq_workspace_bytes.restype = c_size_t
        L.qfp4_gemm_fused_rq_workspace_bytes.argtypes = [c_int64, c_int64, c_int64, c_int]
        L.qfp4_gemm_fused_rq.restype = c_int
        L.qfp4_gemm_fused_rq.argtypes = [P, c_int64, c_int64, c_int, c_int, c_int, P, P, P, c_int64, P, c_size_t,
                                         c_int, P, P]
        L.qfp4_gemm_fused_rq_ex.restype = c_int
        L.qfp4_gemm_fused_rq_ex.argtypes = [P, c_int64, c_int64, c_int, c_int, c_int, P, P, P, P, P, c_int64, P,
                                            c_size_t, c_int, P, P]
        L.qfp4_gemm_fused_rq_workspace_layout.restype = c_int
        L.qfp4_gemm_fused_rq_workspace_layout.argtypes = [c_int64, c_int64, c_int64, c_int, P, P, P]
        L.qfp4_linear_forward_workspace_bytes.restype = c_size_t
        L.qfp4_linear_forward_workspace_bytes.argtypes = [c_int64, c_int64, c_int64, c_int]
        L.qfp4_linear_forward.restype = c_int
        L.qfp4_linear_forward.argtypes = [P, P, c_int64, c_int64, c_int64, c_int, c_int, c_int, P, P, c_size_t, P]
        L.qfp4_linear_backward_workspace_bytes.restype = c_size_t
        L.qfp4_linear_backward_workspace_bytes.argtypes = [c_int64, c_int64, c_int64, c_int]
        L.qfp4_linear_backward.restype = c_int
        L.qfp4_linear_backward.argtypes = [P, P, P, c_int64, c_int64, c_int64, c_int, c_uint64, c_int, P, P, P,
                                           c_size_t, P]
        L.qfp4_gemm_epilogue_workspace_bytes.restype = c_size_t
        L.qfp4_gemm_epilogue_workspace_bytes.argtypes = [c_int64, c_int64, c_int64, c_int]
        L.qfp4_gemm_epilogue.restype = c_int
        L.qfp4_gemm_epilogue.argtypes = [P, P, P, P, P, P, c_int64, c_int64, c_int64, c_int, P, c_int, P, P, c_size_t,
                                         P]
        L.qfp4_linear_forward_epilogue.restype = c_int
        L.qfp4_linear_forward_epilogue.argtypes = [P, P, c_int64, c_int64, c_int64, c_int, c_int, P, c_int, P, P,
                                                   c_size_t, P]
        L.qfp4_epilogue_backward_workspace_bytes.restype = c_size_t
        L.qfp4_epilogue_backward_workspace_bytes.argtypes = [c_int64, c_int64]
        L.qfp4_epilogue_backward.restype = c_int
        L.qfp4_epilogue_backward.argtypes = [P, P, c_int, c_int64, c_int64, c_int, c_double, c_uint64, P, P, P, P,
                                             c_size_t, P]
        L.qfp4_dropout.restype = c_int
        L.qfp4_dropout.argtypes = [P, c_int, c_int64, c_double, c_uint64, P, P, P, P]
        L.qfp4_layernorm_forward.restype = c_int
        L.qfp4_layernorm_forward.argtypes = [P, c_int, c_int64, c_int64, P, P, c_int, c_float, P, P, P, P]
        L.qfp4_layernorm_backward_workspace_bytes.restype = c_size_t
        L.qfp4_layernorm_backward_workspace_bytes.argtypes = [c_int64, c_int64]
        L.qfp4_layernorm_backward.restype = c_int
        L.qfp4_layernorm_backward.argtypes = [P, P, c_int, c_int64, c_int64, P, c_int, P, P, P, P, P, P, c_size_t, P]
        L.qfp4_kl_calibrate_workspace_bytes.restype = c_size_t
        L.qfp4_kl_calibrate_workspace_bytes.argtypes = [c_int, c_int, c_int]
        L.qfp4_kl_calibrate.restype = c_int
        L.qfp4_kl_calibrate.argtypes = [P, c_int, c_int64, c_int, c_int, c_int, P, P, P, P, P, c_size_t, P]
        L.qfp4_status_string.restype = c_char_p
        L.qfp4_status_string.argtypes = [c_int]
        L.qfp4_last_device_error.restype = c_int
        L.qfp4_last_device_error.argtypes = []
        L.qfp4_selftest_wait_timeout.restype = c_int
        L.qfp4_selftest_wait_timeout.argtypes = [c_int64, P]
        L.qfp4_version.restype = c_int
        L.qfp4_version.argtypes = []
        L.qfp4_launch_count.restype = c_uint64
        L.qfp4_launch_count.argtypes = []
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().qfp4_status_string(status).decode()


# ------------------------------------------------------------------ raw C entry points
def qfp4_quantize_workspace_bytes(M, K, fmt, rotate=0, block2d=0):
    return lib().qfp4_quantize_workspace_bytes(M, K, fmt, int(rotate), int(block2d))


def qfp4_quantize(x, xdt, M, K, fmt, rounding, rotate, block2d, four6, seed, codes, scales, codesT, scalesT,
                  tscale, workspace, workspace_bytes, stream):
    return lib().qfp4_quantize(x, xdt, M, K, fmt, rounding, rotate, block2d, four6, seed & ((1 << 64) - 1), codes,
                               scales, codesT, scalesT, tscale, workspace, workspace_bytes, stream)


def qfp4_quantize_ex(x, xdt, M, K, fmt, rounding, rotate, block2d, four6, rule, seed, amax_in, amax_out, codes,
                     scales, codesT, scalesT, tscale, workspace, workspace_bytes, stream):
    return lib().qfp4_quantize_ex(x, xdt, M, K, fmt, rounding, rotate, block2d, four6, rule, seed & ((1 << 64) - 1),
                                  amax_in, amax_out, codes, scales, codesT, scalesT, tscale, workspace,
                                  workspace_bytes, stream)


def qfp4_quantize_mxfp8(x, xdt, M, K, rounding, seed, codes, scales, codesT, scalesT, stream):
    return lib().qfp4_quantize_mxfp8(x, xdt, M, K, rounding, seed & ((1 << 64) - 1), codes, scales, codesT,
                                     scalesT, stream)


def qfp4_quantize_fp32scale(x, xdt, M, K, gran, codes, scales, workspace, workspace_bytes, stream):
    return lib().qfp4_quantize_fp32scale(x, xdt, M, K, gran, codes, scales, workspace, workspace_bytes, stream)


def qfp4_dequantize(codes, scales, tscale, M, K, fmt, out_dt, out, stream):
    return lib().qfp4_dequantize(codes, scales, tscale, M, K, fmt, out_dt, out, stream)


def qfp4_gemm_workspace_bytes(M, N, K, fmt):
    return lib().qfp4_gemm_workspace_bytes(M, N, K, fmt)


def qfp4_gemm_blockscaled(A_codes, A_scales, A_tscale, B_codes, B_scales, B_tscale, M, N, K, fmt, out_dt, out,
                          workspace, workspace_bytes, stream):
    return lib().qfp4_gemm_blockscaled(A_codes, A_scales, A_tscale, B_codes, B_scales, B_tscale, M, N, K, fmt,
                                       out_dt, out, workspace, workspace_bytes, stream)


def qfp4_gemm_blockscaled_noalloc(A_codes, A_scales, A_tscale, B_codes, B_scales, B_tscale, M, N, K, fmt, out_dt,
                                  out, stream):
    """The GEMM without a workspace argument (built-in 16 MiB scratch), for
    callers that may not allocate device memory."""
    return lib().qfp4_gemm_blockscaled_noalloc(A_codes, A_scales, A_tscale, B_codes, B_scales, B_tscale, M, N, K,
                                               fmt, out_dt, out, stream)


def qfp4_gemm_fused_rq_workspace_bytes(M, N, K, fmt):
    return lib().qfp4_gemm_fused_rq_workspace_bytes(M, N, K, fmt)


def qfp4_gemm_fused_rq(A_bf16, M, K, rotate, four6, fmt, B_codes, B_scales, B_tscale, N, workspace,
                       workspace_bytes, out_dt, out, stream):
    return lib().qfp4_gemm_fused_rq(A_bf16, M, K, rotate, four6, fmt, B_codes, B_scales, B_tscale, N, workspace,
                                    workspace_bytes, out_dt, out, stream)


def qfp4_gemm_fused_rq_ex(A_bf16, M, K, rotate, four6, fmt, A_amax_in, A_amax_out, B_codes, B_scales, B_tscale, N,
                          workspace, workspace_bytes, out_dt, out, stream):
    return lib().qfp4_gemm_fused_rq_ex(A_bf16, M, K, rotate, four6, fmt, A_amax_in, A_amax_out, B_codes, B_scales,
                                       B_tscale, N, workspace, workspace_bytes, out_dt, out, stream)


def qfp4_gemm_fused_rq_workspace_layout(M, N, K, fmt):
    """(codes, scales, tscale) byte offsets of A's quantized operand in the
    fused call's workspace."""
    offs = [ctypes.c_size_t() for _ in range(3)]
    st = lib().qfp4_gemm_fused_rq_workspace_layout(M, N, K, fmt, *[ctypes.byref(o) for o in offs])
    _check(st, "qfp4_gemm_fused_rq_workspace_layout")
    return tuple(o.value for o in offs)


def qfp4_linear_forward_workspace_bytes(M, N, K, fmt):
    return lib().qfp4_linear_forward_workspace_bytes(M, N, K, fmt)


def qfp4_linear_forward(X, W, M, N, K, fmt, four6, out_dt, Y, workspace, workspace_bytes, stream):
    return lib().qfp4_linear_forward(X, W, M, N, K, fmt, four6, out_dt, Y, workspace, workspace_bytes, stream)


def qfp4_linear_backward_workspace_bytes(M, N, K, fmt):
    return lib().qfp4_linear_backward_workspace_bytes(M, N, K, fmt)


def qfp4_linear_backward(G, X, W, M, N, K, fmt, seed, out_dt, dX, dW, workspace, workspace_bytes, stream):
    return lib().qfp4_linear_backward(G, X, W, M, N, K, fmt, seed & ((1 << 64) - 1), out_dt, dX, dW, workspace,
                                      workspace_bytes, stream)


def qfp4_gemm_epilogue_workspace_bytes(M, N, K, fmt):
    return lib().qfp4_gemm_epilogue_workspace_bytes(M, N, K, fmt)


def _epilogue_ref(epilogue):
    return None if epilogue is None else ctypes.addressof(epilogue)


def qfp4_gemm_epilogue(A_codes, A_scales, A_tscale, B_codes, B_scales, B_tscale, M, N, K, fmt, epilogue, out_dt, out,
                       workspace, workspace_bytes, stream):
    """epilogue: an ``Epilogue``, or None."""
    return lib().qfp4_gemm_epilogue(A_codes, A_scales, A_tscale, B_codes, B_scales, B_tscale, M, N, K, fmt,
                                    _epilogue_ref(epilogue), out_dt, out, workspace, workspace_bytes, stream)


def qfp4_linear_forward_epilogue(X, W, M, N, K, fmt, four6, epilogue, out_dt, Y, workspace, workspace_bytes, stream):
    """epilogue: an ``Epilogue``, or None."""
    return lib().qfp4_linear_forward_epilogue(X, W, M, N, K, fmt, four6, _epilogue_ref(epilogue), out_dt, Y,
                                              workspace, workspace_bytes, stream)


def qfp4_epilogue_backward_workspace_bytes(M, N):
    return lib().qfp4_epilogue_backward_workspace_bytes(M, N)


def qfp4_epilogue_backward(dY, Z, dt, M, N, act, dropout_p, seed, step, dZ, dbias, workspace, workspace_bytes, stream):
    return lib().qfp4_epilogue_backward(dY, Z, dt, M, N, act, dropout_p, seed & ((1 << 64) - 1), step, dZ, dbias,
                                        workspace, workspace_bytes, stream)


def qfp4_dropout(x, dt, n, p, seed, step, residual, out, stream):
    return lib().qfp4_dropout(x, dt, n, p, seed & ((1 << 64) - 1), step, residual, out, stream)


def qfp4_layernorm_forward(x, dt, M, D, gamma, beta, wdt, eps, y, mean, rstd, stream):
    return lib().qfp4_layernorm_forward(x, dt, M, D, gamma, beta, wdt, eps, y, mean, rstd, stream)


def qfp4_layernorm_backward_workspace_bytes(M, D):
    return lib().qfp4_layernorm_backward_workspace_bytes(M, D)


def qfp4_layernorm_backward(dy, x, dt, M, D, gamma, wdt, mean, rstd, dx, dgamma, dbeta, workspace, workspace_bytes,
                            stream):
    return lib().qfp4_layernorm_backward(dy, x, dt, M, D, gamma, wdt, mean, rstd, dx, dgamma, dbeta, workspace,
                                         workspace_bytes, stream)


def qfp4_kl_calibrate_workspace_bytes(bins, levels, grid):
    return lib().qfp4_kl_calibrate_workspace_bytes(bins, levels, grid)


def qfp4_kl_calibrate(x, xdt, n, bins, levels, grid, clip_out, best_bins_out, kl_out, hist_out, workspace,
                      workspace_bytes, stream):
    return lib().qfp4_kl_calibrate(x, xdt, n, bins, levels, grid, clip_out, best_bins_out, kl_out, hist_out,
                                   workspace, workspace_bytes, stream)


def qfp4_status_string(status):
    return status_string(status)


def qfp4_last_device_error():
    return lib().qfp4_last_device_error()


def qfp4_selftest_wait_timeout(limit_us, stream):
    return lib().qfp4_selftest_wait_timeout(limit_us, stream)


def qfp4_version():
    return lib().qfp4_version()


def qfp4_launch_count():
    return lib().qfp4_launch_count()


# ------------------------------------------------------------------ torch conveniences
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _xdt(x):
    torch = _torch()
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise TypeError("x must be bfloat16 or float32")


def _check(st, where):
    if st != OK:
        raise QFP4Error(st, where)


def _input(t, name, dims=2):
    """An input tensor the C ABI can read as a plain pointer: on a CUDA
    device, contiguous (row-major), with `dims` dimensions (None: any)."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")


def quantize(x, fmt=MXFP4, rounding=RNE, rotate=False, block2d=False, four6=False, seed=0, transposed=False,
             stream=None, out=None, workspace=None, rule=SCALE_DEFAULT, amax_in=None, amax_out=None):
    """Quantize a contiguous (M, K) bf16/fp32 CUDA tensor; returns a dict of
    uint8 codes (M, K/2), scales (M, K/g), optional codesT/scalesT, and the
    float32 tscale (NVFP4).  ``out`` may supply preallocated buffers.
    ``rule``, ``amax_in`` / ``amax_out`` (one-element float32 CUDA tensors)
    are qfp4_quantize_ex's scale rule and tensor-amax options."""
    torch = _torch()
    _input(x, "x")
    M, K = x.shape
    g = 32 if fmt == MXFP4 else 16
    dev = x.device
    o = dict(out) if out is not None else {}
    if "codes" not in o:
        o["codes"] = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
        o["scales"] = torch.empty((M, K // g), dtype=torch.uint8, device=dev)
        if transposed:
            o["codesT"] = torch.empty((K, M // 2), dtype=torch.uint8, device=dev)
            o["scalesT"] = torch.empty((K, M // g), dtype=torch.uint8, device=dev)
        if fmt == NVFP4:
            o["tscale"] = torch.empty(1, dtype=torch.float32, device=dev)
    wsb = qfp4_quantize_workspace_bytes(M, K, fmt, rotate, block2d)
    if workspace is None and wsb:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    st = qfp4_quantize_ex(_ptr(x), _xdt(x), M, K, fmt, rounding, int(rotate), int(block2d), int(four6), rule, seed,
                          _ptr(amax_in), _ptr(amax_out), _ptr(o["codes"]), _ptr(o["scales"]), _ptr(o.get("codesT")),
                          _ptr(o.get("scalesT")), _ptr(o.get("tscale")), _ptr(workspace), wsb, _stream(stream))
    _check(st, "qfp4_quantize_ex")
    return o


def quantize_mxfp8(x, rounding=RNE, seed=0, transposed=False, stream=None, out=None):
    torch = _torch()
    _input(x, "x")
    M, K = x.shape
    dev = x.device
    o = dict(out) if out is not None else {}
    if "codes" not in o:
        o["codes"] = torch.empty((M, K), dtype=torch.uint8, device=dev)
        o["scales"] = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
        if transposed:
            o["codesT"] = torch.empty((K, M), dtype=torch.uint8, device=dev)
            o["scalesT"] = torch.empty((K, M // 32), dtype=torch.uint8, device=dev)
    st = qfp4_quantize_mxfp8(_ptr(x), _xdt(x), M, K, rounding, seed, _ptr(o["codes"]), _ptr(o["scales"]),
                             _ptr(o.get("codesT")), _ptr(o.get("scalesT")), _stream(stream))
    _check(st, "qfp4_quantize_mxfp8")
    return o


def quantize_fp32scale(x, gran, stream=None, out=None):
    torch = _torch()
    _input(x, "x")
    M, K = x.shape
    dev = x.device
    n_scales = {GRAN_TENSOR: 1, GRAN_ROW: M, GRAN_GROUP16: M * K // 16, GRAN_GROUP32: M * K // 32}[gran]
    o = dict(out) if out is not None else {
        "codes": torch.empty((M, K // 2), dtype=torch.uint8, device=dev),
        "scales": torch.empty(n_scales, dtype=torch.float32, device=dev)}
    wsb = qfp4_quantize_workspace_bytes(M, K, NVFP4)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
    st = qfp4_quantize_fp32scale(_ptr(x), _xdt(x), M, K, gran, _ptr(o["codes"]), _ptr(o["scales"]), _ptr(ws), wsb,
                                 _stream(stream))
    _check(st, "qfp4_quantize_fp32scale")
    return o


def dequantize(q, M, K, fmt, out_dtype=None, stream=None, out=None):
    torch = _torch()
    if out is None:
        out_dtype = torch.float32 if out_dtype is None else out_dtype
        out = torch.empty((M, K), dtype=out_dtype, device=q["codes"].device)
    out_dtype = out.dtype
    st = qfp4_dequantize(_ptr(q["codes"]), _ptr(q["scales"]), _ptr(q.get("tscale")), M, K, fmt,
                         F32 if out_dtype == torch.float32 else BF16, _ptr(out), _stream(stream))
    _check(st, "qfp4_dequantize")
    return out


def gemm(A, B, M, N, K, fmt, out_dtype=None, out=None, workspace=None, stream=None):
    """Y = deq(A) deq(B)^T for operands as returned by ``quantize``."""
    torch = _torch()
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A["codes"].device)
    wsb = qfp4_gemm_workspace_bytes(M, N, K, fmt)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=A["codes"].device)
    st = qfp4_gemm_blockscaled(_ptr(A["codes"]), _ptr(A["scales"]), _ptr(A.get("tscale")), _ptr(B["codes"]),
                               _ptr(B["scales"]), _ptr(B.get("tscale")), M, N, K, fmt,
                               F32 if out.dtype == torch.float32 else BF16, _ptr(out), _ptr(workspace), wsb,
                               _stream(stream))
    _check(st, "qfp4_gemm_blockscaled")
    return out


def gemm_fused_rq(A_bf16, B, N, fmt=NVFP4, rotate=True, four6=False, out_dtype=None, out=None, workspace=None,
                  stream=None, A_amax_in=None, A_amax_out=None):
    """Y = Q(rot(A)) deq(B)^T with A bf16 (M, K) quantized inside the call;
    A_amax_in / A_amax_out: NVFP4 tensor amax of A supplied / reported
    (one-element float32 CUDA tensors)."""
    torch = _torch()
    _input(A_bf16, "A_bf16")
    M, K = A_bf16.shape
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A_bf16.device)
    wsb = qfp4_gemm_fused_rq_workspace_bytes(M, N, K, fmt)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=A_bf16.device)
    st = qfp4_gemm_fused_rq_ex(_ptr(A_bf16), M, K, int(rotate), int(four6), fmt, _ptr(A_amax_in), _ptr(A_amax_out),
                               _ptr(B["codes"]), _ptr(B["scales"]), _ptr(B.get("tscale")), N, _ptr(workspace), wsb,
                               F32 if out.dtype == torch.float32 else BF16, _ptr(out), _stream(stream))
    _check(st, "qfp4_gemm_fused_rq_ex")
    return out


def linear_forward(X, W, fmt=NVFP4, four6=False, out_dtype=None, out=None, workspace=None, stream=None):
    """Y = X W^T through rotated FP4 operands (qfp4_linear_forward); X (M, K)
    and W (N, K) bf16 CUDA tensors."""
    torch = _torch()
    _input(X, "X")
    _input(W, "W")
    M, K = X.shape
    N = W.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32 if out_dtype is None else out_dtype, device=X.device)
    wsb = qfp4_linear_forward_workspace_bytes(M, N, K, fmt)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=X.device)
    st = qfp4_linear_forward(_ptr(X), _ptr(W), M, N, K, fmt, int(four6), F32 if out.dtype == torch.float32 else BF16,
                             _ptr(out), _ptr(workspace), wsb, _stream(stream))
    _check(st, "qfp4_linear_forward")
    return out


def linear_backward(G, X, W, fmt=NVFP4, seed=0, out_dtype=None, want_dx=True, want_dw=True, out=None,
                    workspace=None, stream=None):
    """(dX, dW) = (G W, G^T X) through quantized operands
    (qfp4_linear_backward); G (M, N), X (M, K), W (N, K) bf16 CUDA tensors."""
    torch = _torch()
    _input(G, "G")
    for t, name in ((X, "X"), (W, "W")):
        if t is not None:
            _input(t, name)
    M, N = G.shape
    K = X.shape[1] if X is not None else W.shape[1]
    dt = torch.float32 if out_dtype is None else out_dtype
    o = dict(out) if out is not None else {}
    if want_dx and "dX" not in o:
        o["dX"] = torch.empty((M, K), dtype=dt, device=G.device)
    if want_dw and "dW" not in o:
        o["dW"] = torch.empty((N, K), dtype=dt, device=G.device)
    wsb = qfp4_linear_backward_workspace_bytes(M, N, K, fmt)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=G.device)
    st = qfp4_linear_backward(_ptr(G), _ptr(X), _ptr(W), M, N, K, fmt, seed, F32 if dt == torch.float32 else BF16,
                              _ptr(o.get("dX")), _ptr(o.get("dW")), _ptr(workspace), wsb, _stream(stream))
    _check(st, "qfp4_linear_backward")
    return o.get("dX"), o.get("dW")


# ------------------------------------------------------------------ around a linear layer
# These wrappers check every tensor they hand over; a call on a few rows costs
# about as much in Python as on the device, so the checks are one expression
# where they pass and name the fault only where they fail.
_current_device = None      # the current device's index
_raw_stream = None          # device index -> handle of its current stream


def _cuda_api():
    global _current_device, _raw_stream
    torch = _torch()
    _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _tensor(t, name, index, shape=None, dtype=None):
    """Checks of a tensor that goes to the C ABI: CUDA, contiguous, on device
    `index`, and of the given shape and dtype; its address."""
    if not (t.is_cuda and t.is_contiguous() and t.get_device() == index and (shape is None or t.shape == shape)
            and (dtype is None or t.dtype is dtype)):
        _input(t, name, dims=None)
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, not {t.device}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t.data_ptr()


def _param(t, name, index, shape):
    """(address, C type) of a bf16 or fp32 parameter, or (None, BF16)."""
    if t is None:
        return None, BF16
    torch = _torch()
    p = _tensor(t, name, index, shape)
    if t.dtype is torch.bfloat16:
        return p, BF16
    if t.dtype is torch.float32:
        return p, F32
    raise TypeError(f"{name} must be bfloat16 or float32")


def _step(step, index):
    """The dropout's step counter: None, or a one-element int64 CUDA tensor."""
    if step is None:
        return None
    p = _tensor(step, "step", index, None, _torch().int64)
    if step.numel() != 1:
        raise ValueError("step must have one element")
    return p


def _new(like, stream, dtype, *shape):
    """A fresh tensor on `like`'s device, of the allocator's pool for the
    stream that the call runs on (its memory may still be in use elsewhere
    on any other)."""
    if stream is None:
        return _torch().empty(*shape, dtype=dtype, device=like.device)
    with _torch().cuda.stream(stream):
        return _torch().empty(*shape, dtype=dtype, device=like.device)


def _new_like(like, stream):
    """The same with `like`'s shape and type (contiguous, as `like` is)."""
    if stream is None:
        return _torch().empty_like(like)
    with _torch().cuda.stream(stream):
        return _torch().empty_like(like)


def _call(fn, index, stream, *args):
    """fn(*args, stream) on device `index` (the C ABI launches on the current
    one) and `stream` (default: that device's current stream)."""
    if _raw_stream is None:
        _cuda_api()
    if _current_device() == index:
        st = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with _torch().cuda.device(index):
            st = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if st != OK:
        raise QFP4Error(st, fn.__name__)


_gemm_epilogue_ws = functools.lru_cache(1024)(qfp4_gemm_epilogue_workspace_bytes)
_linear_forward_ws = functools.lru_cache(1024)(qfp4_linear_forward_workspace_bytes)
_epilogue_backward_ws = functools.lru_cache(1024)(qfp4_epilogue_backward_workspace_bytes)
_layernorm_backward_ws = functools.lru_cache(1024)(qfp4_layernorm_backward_workspace_bytes)


def _scratch(workspace, nbytes, like, stream):
    """(address, bytes, the tensor that has to live until the call) of the
    caller's workspace, or of a fresh one."""
    if workspace is not None:
        return _tensor(workspace, "workspace", like.get_device()), workspace.nbytes, workspace
    if not nbytes:
        return None, 0, None
    workspace = _new(like, stream, _torch().uint8, nbytes)
    return workspace.data_ptr(), nbytes, workspace


def _operand(q, name, rows, K, fmt, index):
    """Addresses of codes, scales and tensor scale."""
    torch = _torch()
    u8 = torch.uint8
    c = _tensor(q["codes"], f"{name} codes", index, (rows, K if fmt == MXFP8 else K // 2), u8)
    s = _tensor(q["scales"], f"{name} scales", index, (rows, K // (16 if fmt == NVFP4 else 32)), u8)
    return c, s, _tensor(q["tscale"], f"{name} tscale", index, None, torch.float32) if fmt == NVFP4 else None


def _output(out, shape, out_dtype, like, index, stream):
    """(tensor, address, C type) of a bf16 or fp32 output."""
    torch = _torch()
    if out is None:
        out = _new(like, stream, torch.float32 if out_dtype is None else out_dtype, *shape)
        p = out.data_ptr()
    else:
        p = _tensor(out, "out", index, shape)
    if out.dtype is torch.float32:
        return out, p, F32
    if out.dtype is torch.bfloat16:
        return out, p, BF16
    raise TypeError("outputs are bfloat16 or float32")


def _epilogue(shape, out, index, bias, act, want_preact, dropout_p, seed, step, residual, stream):
    """(Epilogue struct, preact tensor or None) for an output tensor."""
    e = Epilogue()
    e.act = act
    if bias is not None:
        e.bias, e.bias_dt = _param(bias, "bias", index, shape[1:])
    if residual is not None:
        e.residual, e.residual_dt = _param(residual, "residual", index, shape)
    preact = None
    if want_preact is True:
        preact = _new_like(out, stream)
        e.preact = preact.data_ptr()
    elif want_preact is not False and want_preact is not None:
        preact = want_preact
        e.preact = _tensor(preact, "preact", index, shape, out.dtype)
    if dropout_p or step is not None:
        e.dropout_p, e.seed, e.step = dropout_p, seed & ((1 << 64) - 1), _step(step, index)
    return e, preact


def gemm_epilogue(A, B, M, N, K, fmt, bias=None, act=ACT_NONE, want_preact=False, dropout_p=0.0, seed=0, step=None,
                  residual=None, out_dtype=None, out=None, workspace=None, stream=None):
    """(Y, preact) with Y = residual + dropout(act(deq(A) deq(B)^T + bias)) in
    one GEMM (qfp4_gemm_epilogue), for operands as returned by ``quantize`` or
    ``quantize_mxfp8``.  ``want_preact``: True (or a buffer) to keep the sum
    before the activation for ``epilogue_backward``, else preact is None.
    ``step``: a one-element int64 CUDA tensor, the dropout's counter."""
    like = B["codes"]
    _input(like, "B codes")
    index = like.get_device()
    ac, sa, ta = _operand(A, "A", M, K, fmt, index)
    bc, sb, tb = _operand(B, "B", N, K, fmt, index)
    shape = (M, N)
    out, po, dt = _output(out, shape, out_dtype, like, index, stream)
    e, preact = _epilogue(shape, out, index, bias, act, want_preact, dropout_p, seed, step, residual, stream)
    ws, wsb, keep = _scratch(workspace, _gemm_epilogue_ws(M, N, K, fmt), like, stream)
    _call(qfp4_gemm_epilogue, index, stream, ac, sa, ta, bc, sb, tb, M, N, K, fmt, e, dt, po, ws, wsb)
    return out, preact


def linear_forward_epilogue(X, W, fmt=NVFP4, four6=False, bias=None, act=ACT_NONE, want_preact=False, dropout_p=0.0,
                            seed=0, step=None, residual=None, out_dtype=None, out=None, workspace=None, stream=None):
    """``linear_forward`` with the epilogue of ``gemm_epilogue``
    (qfp4_linear_forward_epilogue); returns (Y, preact)."""
    bf16 = _torch().bfloat16
    _input(X, "X")
    _input(W, "W")
    index = X.get_device()
    M, K = X.shape
    N = W.shape[0]
    px, pw = _tensor(X, "X", index, None, bf16), _tensor(W, "W", index, (N, K), bf16)
    shape = (M, N)
    out, po, dt = _output(out, shape, out_dtype, X, index, stream)
    e, preact = _epilogue(shape, out, index, bias, act, want_preact, dropout_p, seed, step, residual, stream)
    ws, wsb, keep = _scratch(workspace, _linear_forward_ws(M, N, K, fmt), X, stream)
    _call(qfp4_linear_forward_epilogue, index, stream, px, pw, M, N, K, fmt, int(four6), e, dt, po, ws, wsb)
    return out, preact


def epilogue_backward(dY, Z=None, act=ACT_NONE, dropout_p=0.0, seed=0, step=None, want_dbias=True, out=None,
                      workspace=None, stream=None):
    """(dZ, dbias) of an epilogue's dropout, activation and bias
    (qfp4_epilogue_backward): dY (M, N) and the forward's preact Z, bf16 or
    fp32; dZ of their type, dbias (N,) fp32 or None.  ``out`` may supply a
    dict with dZ and dbias."""
    _input(dY, "dY")
    index, shape, dtype = dY.get_device(), dY.shape, dY.dtype
    M, N = shape
    dt = _xdt(dY)
    pz = None if Z is None else _tensor(Z, "Z", index, shape, dtype)
    dZ = db = pd = pb = ws = keep = None
    wsb = 0
    if out is not None:
        dZ, db = out.get("dZ"), out.get("dbias")
        pd = None if dZ is None else _tensor(dZ, "dZ", index, shape, dtype)
        pb = None if db is None else _tensor(db, "dbias", index, (N,), _torch().float32)
    if dZ is None:
        dZ = _new_like(dY, stream)
        pd = dZ.data_ptr()
    if db is None and want_dbias:
        db = _new(dY, stream, _torch().float32, N)
        pb = db.data_ptr()
    if db is not None:
        ws, wsb, keep = _scratch(workspace, _epilogue_backward_ws(M, N), dY, stream)
    _call(qfp4_epilogue_backward, index, stream, dY.data_ptr(), pz, dt, M, N, act, dropout_p, seed,
          _step(step, index), pd, pb, ws, wsb)
    return dZ, db


def dropout(x, p, seed=0, step=None, residual=None, out=None, stream=None):
    """x / (1 - p) where the Philox word of an element lets it stay, else 0,
    plus the residual (qfp4_dropout); x bf16 or fp32 of any shape.  The same
    call on the output's gradient is the backward pass."""
    _input(x, "x", dims=None)
    index = x.get_device()
    dt = _xdt(x)
    pr = None if residual is None else _tensor(residual, "residual", index, x.shape, x.dtype)
    if out is None:
        out = _new_like(x, stream)
        po = out.data_ptr()
    else:
        po = _tensor(out, "out", index, x.shape, x.dtype)
    _call(qfp4_dropout, index, stream, x.data_ptr(), dt, x.numel(), p, seed, _step(step, index), pr, po)
    return out


def _norm_params(index, D, gamma, beta):
    """(gamma's address, beta's, their one C type)."""
    pg, gdt = _param(gamma, "gamma", index, (D,))
    pb, bdt = _param(beta, "beta", index, (D,))
    if gamma is not None and beta is not None and gdt != bdt:
        raise TypeError("gamma and beta must have one dtype")
    return pg, pb, bdt if gamma is None else gdt


def layernorm_forward(x, gamma=None, beta=None, eps=1e-5, want_stats=True, out=None, stream=None):
    """(y, mean, rstd) of the rows of x (M, D), bf16 or fp32
    (qfp4_layernorm_forward); gamma and beta (D,) bf16 or fp32, or None; mean
    and rstd (M,) fp32, or None without ``want_stats``.  ``out`` may supply a
    dict with y, mean and rstd."""
    _input(x, "x")
    index, shape = x.get_device(), x.shape
    M, D = shape
    dt = _xdt(x)
    pg, pb, wdt = _norm_params(index, D, gamma, beta)
    f32 = _torch().float32
    if out is None:
        y = _new_like(x, stream)
        py, mean, rstd, pm, pr = y.data_ptr(), None, None, None, None
        if want_stats:
            mean = _new(x, stream, f32, M)
            rstd = _new_like(mean, stream)
            pm, pr = mean.data_ptr(), rstd.data_ptr()
    else:
        y, mean, rstd = out.get("y"), out.get("mean"), out.get("rstd")
        if y is None:
            y = _new_like(x, stream)
        if mean is None and want_stats:
            mean = _new(x, stream, f32, M)
        if rstd is None and want_stats:
            rstd = _new(x, stream, f32, M)
        py = _tensor(y, "y", index, shape, x.dtype)
        pm = None if mean is None else _tensor(mean, "mean", index, (M,), f32)
        pr = None if rstd is None else _tensor(rstd, "rstd", index, (M,), f32)
    _call(qfp4_layernorm_forward, index, stream, x.data_ptr(), dt, M, D, pg, pb, wdt, eps, py, pm, pr)
    return y, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd, want_dx=True, want_dw=True, out=None, workspace=None, stream=None):
    """(dx, dgamma, dbeta) of ``layernorm_forward`` (qfp4_layernorm_backward);
    dx of x's type, dgamma and dbeta (D,) fp32; None for what is not wanted.
    ``out`` may supply a dict with dx, dgamma and dbeta."""
    _input(x, "x")
    index, shape, dtype = x.get_device(), x.shape, x.dtype
    M, D = shape
    dt = _xdt(x)
    f32 = _torch().float32
    pg, _, wdt = _norm_params(index, D, gamma, None)
    py = _tensor(dy, "dy", index, shape, dtype)
    pm, pr = _tensor(mean, "mean", index, (M,), f32), _tensor(rstd, "rstd", index, (M,), f32)
    dx = dg = db = px = pdg = pdb = ws = keep = None
    wsb = 0
    if out is not None:
        dx, dg, db = out.get("dx"), out.get("dgamma"), out.get("dbeta")
        px = None if dx is None else _tensor(dx, "dx", index, shape, dtype)
        pdg = None if dg is None else _tensor(dg, "dgamma", index, (D,), f32)
        pdb = None if db is None else _tensor(db, "dbeta", index, (D,), f32)
    if dx is None and want_dx:
        dx = _new_like(x, stream)
        px = dx.data_ptr()
    if dg is None and want_dw:
        dg = _new(x, stream, f32, D)
        pdg = dg.data_ptr()
    if db is None and want_dw:
        db = _new_like(dg, stream)
        pdb = db.data_ptr()
    if dg is not None or db is not None:
        ws, wsb, keep = _scratch(workspace, _layernorm_backward_ws(M, D), x, stream)
    _call(qfp4_layernorm_backward, index, stream, py, x.data_ptr(), dt, M, D, pg, wdt, pm, pr, px, pdg, pdb, ws, wsb)
    return dx, dg, db


def kl_calibrate(x, bins=2048, levels=8, grid=0, stream=None, out=None):
    """KL-divergence clip point of a CUDA tensor (qfp4_kl_calibrate); returns
    dict(clip (1,) float32, best (1,) int32, kl (bins - first + 1,) float64,
    hist (bins,) int64 holding the uint64 counts)."""
    torch = _torch()
    _input(x, "x", dims=None)
    dev = x.device
    first = 8 if grid else levels
    o = dict(out) if out is not None else {
        "clip": torch.empty(1, dtype=torch.float32, device=dev), "best": torch.empty(1, dtype=torch.int32, device=dev),
        "kl": torch.empty(bins - first + 1, dtype=torch.float64, device=dev),
        "hist": torch.empty(bins, dtype=torch.int64, device=dev)}
    wsb = qfp4_kl_calibrate_workspace_bytes(bins, levels, grid)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    st = qfp4_kl_calibrate(_ptr(x), _xdt(x), x.numel(), bins, levels, grid, _ptr(o["clip"]), _ptr(o["best"]),
                           _ptr(o["kl"]), _ptr(o["hist"]), _ptr(ws), wsb, _stream(stream))
    _check(st, "qfp4_kl_calibrate")
    return o

