"""Thin Python binding of libnvfp4.so (ctypes).

The functions named ``nvfp4_*`` mirror the C ABI in include/nvfp4.h one to
one: arguments are marshalled (torch tensors -> device pointers, the current
torch stream -> cudaStream_t) and the status is turned into an exception.
Every step of the NVFP4 path runs in the library's CUDA kernels; there is no
fallback of any kind -- if the library cannot be loaded, calls raise.

The lower-case helpers (``quantize_1d`` ...) only allocate the outputs with
torch (PyTorch is used for device memory and streams) and call the C ABI.
With ``stream`` (a torch stream or a handle) a helper allocates and launches
there; its tensors may be dropped on either stream at any time.  What orders
the two streams, as ever, is the caller's wait on one for the other.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

NVFP4_OK = 0
(NVFP4_ERR_INVALID_ARG, NVFP4_ERR_UNSUPPORTED_SHAPE, NVFP4_ERR_MISALIGNED, NVFP4_ERR_CUDA, NVFP4_ERR_TIMEOUT,
 NVFP4_ERR_WORKSPACE) = 1, 2, 3, 4, 5, 6
NVFP4_RNE, NVFP4_SR = 0, 1
NVFP4_SCALE_1D, NVFP4_SCALE_2D = 0, 1
NVFP4_OUT_F32, NVFP4_OUT_BF16 = 0, 1
(NVFP4_ACT_NONE, NVFP4_ACT_RELU, NVFP4_ACT_RELU2, NVFP4_ACT_GELU, NVFP4_ACT_GELU_TANH, NVFP4_ACT_SILU) = range(6)

EXPORTS = (
    "nvfp4_version", "nvfp4_status_string", "nvfp4_workspace_size", "nvfp4_mma_scale_bytes",
    "nvfp4_quantize_1d", "nvfp4_rht_quantize_sr", "nvfp4_quantize_2d", "nvfp4_dequantize", "nvfp4_gemm",
    "nvfp4_scales_to_mma", "nvfp4_kernel_launches", "nvfp4_get_error", "nvfp4_quantize_1d_noalloc",
    "nvfp4_selftest_wait_timeout", "nvfp4_quantize_1d_from_amax", "nvfp4_quantize_2d_from_amax",
    "nvfp4_gemm_amax", "nvfp4_mxfp4_quantize", "nvfp4_mxfp4_dequantize", "nvfp4_mxfp4_gemm",
    "nvfp4_quantize_dual", "nvfp4_rht_quantize_n", "nvfp4_gemm_epilogue", "nvfp4_act_grad_workspace_size",
    "nvfp4_act_grad", "nvfp4_moe_rows", "nvfp4_moe_workspace_size", "nvfp4_moe_sort", "nvfp4_moe_gather",
    "nvfp4_moe_combine", "nvfp4_moe_combine_grad", "nvfp4_gemm_grouped", "nvfp4_gemm_grouped_wgrad",
)

_lib = None
_current_device = torch._C._cuda_getDevice


class Nvfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {lib().nvfp4_status_string(status).decode()} (status {status})")


def lib():
    """Load libnvfp4.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"libnvfp4.so not built (expected at {LIB_PATH}); run "
                          "`python -m nvfp4_bit_block_amax_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, u64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_size_t
        L.nvfp4_version.restype = ci
        L.nvfp4_version.argtypes = []
        L.nvfp4_status_string.restype = ctypes.c_char_p
        L.nvfp4_status_string.argtypes = [ci]
        L.nvfp4_workspace_size.restype = sz
        L.nvfp4_workspace_size.argtypes = [i64, i64]
        L.nvfp4_mma_scale_bytes.restype = sz
        L.nvfp4_mma_scale_bytes.argtypes = [i64, i64]
        L.nvfp4_quantize_1d.restype = ci
        L.nvfp4_quantize_1d.argtypes = [vp, i64, i64, i64, ci, ci, u64, vp, vp, vp, vp, vp, sz, vp]
        L.nvfp4_quantize_1d_noalloc.restype = ci
        L.nvfp4_quantize_1d_noalloc.argtypes = [vp, i64, i64, i64, ci, ci, u64, vp, vp, vp, vp, vp]
        L.nvfp4_rht_quantize_sr.restype = ci
        L.nvfp4_rht_quantize_sr.argtypes = [vp, i64, i64, i64, ci, u64, ci, u64, vp, vp, vp, vp, vp, sz, vp]
        L.nvfp4_rht_quantize_n.restype = ci
        L.nvfp4_rht_quantize_n.argtypes = [vp, i64, i64, i64, ci, ci, u64, ci, u64, vp, vp, vp, vp, vp, sz, vp]
        L.nvfp4_quantize_2d.restype = ci
        L.nvfp4_quantize_2d.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.nvfp4_dequantize.restype = ci
        L.nvfp4_dequantize.argtypes = [vp, vp, ci, vp, i64, i64, ci, vp, vp]
        L.nvfp4_gemm.restype = ci
        L.nvfp4_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, i64, vp]
        L.nvfp4_scales_to_mma.restype = ci
        L.nvfp4_scales_to_mma.argtypes = [vp, ci, i64, i64, vp, vp]
        L.nvfp4_kernel_launches.restype = ctypes.c_longlong
        L.nvfp4_kernel_launches.argtypes = []
        L.nvfp4_get_error.restype = ci
        L.nvfp4_get_error.argtypes = [vp]
        L.nvfp4_selftest_wait_timeout.restype = ci
        L.nvfp4_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        L.nvfp4_quantize_1d_from_amax.restype = ci
        L.nvfp4_quantize_1d_from_amax.argtypes = [vp, i64, i64, i64, ci, ci, u64, vp, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_2d_from_amax.restype = ci
        L.nvfp4_quantize_2d_from_amax.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.nvfp4_gemm_amax.restype = ci
        L.nvfp4_gemm_amax.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, i64, vp, vp]
        L.nvfp4_mxfp4_quantize.restype = ci
        L.nvfp4_mxfp4_quantize.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
        L.nvfp4_mxfp4_dequantize.restype = ci
        L.nvfp4_mxfp4_dequantize.argtypes = [vp, vp, i64, i64, ci, vp, vp]
        L.nvfp4_quantize_dual.restype = ci
        L.nvfp4_quantize_dual.argtypes = [vp, i64, i64, i64, ci, u64, vp, vp, vp, vp, u64, u64, vp, vp, vp, vp, vp,
                                          sz, vp]
        L.nvfp4_mxfp4_gemm.restype = ci
        L.nvfp4_mxfp4_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, vp, i64, vp]
        L.nvfp4_gemm_epilogue.restype = ci
        L.nvfp4_gemm_epilogue.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, ci, vp, i64, ci, vp, i64, vp, i64,
                                          vp, vp]
        L.nvfp4_act_grad_workspace_size.restype = sz
        L.nvfp4_act_grad_workspace_size.argtypes = [i64, i64]
        L.nvfp4_act_grad.restype = ci
        L.nvfp4_act_grad.argtypes = [vp, i64, vp, i64, i64, i64, ci, vp, vp, i64, vp, i64, vp, vp, vp, sz, vp]
        L.nvfp4_moe_rows.restype = i64
        L.nvfp4_moe_rows.argtypes = [i64, i64]
        L.nvfp4_moe_workspace_size.restype = sz
        L.nvfp4_moe_workspace_size.argtypes = [i64, i64]
        L.nvfp4_moe_sort.restype = ci
        L.nvfp4_moe_sort.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp]
        L.nvfp4_moe_gather.restype = ci
        L.nvfp4_moe_gather.argtypes = [vp, i64, i64, i64, i64, vp, vp, i64, vp, i64, vp, vp]
        L.nvfp4_moe_combine.restype = ci
        L.nvfp4_moe_combine.argtypes = [vp, i64, i64, i64, vp, vp, vp, i64, i64, i64, vp, i64, vp]
        L.nvfp4_moe_combine_grad.restype = ci
        L.nvfp4_moe_combine_grad.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, vp, i64, vp, vp, i64, vp, vp, vp]
        L.nvfp4_gemm_grouped.restype = ci
        L.nvfp4_gemm_grouped.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, ci, vp, i64, ci, vp,
                                         i64, vp, i64, vp, vp]
        L.nvfp4_gemm_grouped_wgrad.restype = ci
        L.nvfp4_gemm_grouped_wgrad.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, ci, vp, i64, vp]
        _lib = L
    return _lib


def _p(t) -> Optional[int]:
    """Device pointer of a tensor (None / int pass through)."""
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:   # the current stream's handle, without building a Stream object (3 us a call)
        return torch._C._cuda_getCurrentRawStream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != NVFP4_OK:
        raise Nvfp4Error(fn, status)


# ------------------------------------------------------------- C ABI mirror --
def nvfp4_version() -> int:
    return lib().nvfp4_version()


def nvfp4_status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()


def nvfp4_workspace_size(rows: int, cols: int) -> int:
    return lib().nvfp4_workspace_size(rows, cols)


def nvfp4_mma_scale_bytes(rows: int, k: int) -> int:
    return lib().nvfp4_mma_scale_bytes(rows, k)


def nvfp4_kernel_launches() -> int:
    return lib().nvfp4_kernel_launches()


def nvfp4_quantize_1d(x, rows, cols, ld, transpose, rounding, sr_seed, codes, scales, scales_mma,
                      global_scale, workspace, ws_bytes, stream=None):
    _check("nvfp4_quantize_1d", lib().nvfp4_quantize_1d(
        _p(x), rows, cols, ld, transpose, rounding, sr_seed, _p(codes), _p(scales), _p(scales_mma),
        _p(global_scale), _p(workspace), ws_bytes, _stream(stream)))


def nvfp4_quantize_1d_noalloc(x, rows, cols, ld, transpose, rounding, sr_seed, codes, scales, scales_mma,
                              global_scale, stream=None):
    """nvfp4_quantize_1d without a workspace argument: for callers that cannot
    allocate device memory, the library uses its own static scratch."""
    _check("nvfp4_quantize_1d_noalloc", lib().nvfp4_quantize_1d_noalloc(
        _p(x), rows, cols, ld, transpose, rounding, sr_seed, _p(codes), _p(scales), _p(scales_mma),
        _p(global_scale), _stream(stream)))


def nvfp4_rht_quantize_sr(x, rows, cols, ld, transpose, rht_seed, rounding, sr_seed, codes, scales, scales_mma,
                          global_scale, workspace, ws_bytes, stream=None):
    _check("nvfp4_rht_quantize_sr", lib().nvfp4_rht_quantize_sr(
        _p(x), rows, cols, ld, transpose, rht_seed, rounding, sr_seed, _p(codes), _p(scales), _p(scales_mma),
        _p(global_scale), _p(workspace), ws_bytes, _stream(stream)))


def nvfp4_rht_quantize_n(x, rows, cols, ld, transpose, rht_order, rht_seed, rounding, sr_seed, codes, scales,
                         scales_mma, global_scale, workspace, ws_bytes, stream=None):
    _check("nvfp4_rht_quantize_n", lib().nvfp4_rht_quantize_n(
        _p(x), rows, cols, ld, transpose, rht_order, rht_seed, rounding, sr_seed, _p(codes), _p(scales),
        _p(scales_mma), _p(global_scale), _p(workspace), ws_bytes, _stream(stream)))


def nvfp4_quantize_dual(x, rows, cols, ld, rounding, sr_seed, codes, scales, scales_mma, global_scale, rht_seed,
                        sr_seed_t, codes_t, scales_t, scales_mma_t, global_scale_t, workspace, ws_bytes, stream=None):
    _check("nvfp4_quantize_dual", lib().nvfp4_quantize_dual(
        _p(x), rows, cols, ld, rounding, sr_seed, _p(codes), _p(scales), _p(scales_mma), _p(global_scale), rht_seed,
        sr_seed_t, _p(codes_t), _p(scales_t), _p(scales_mma_t), _p(global_scale_t), _p(workspace), ws_bytes,
        _stream(stream)))


def nvfp4_quantize_2d(w, rows, cols, ld, codes_row, codes_col, scales, scales_mma_row, scales_mma_col,
                      global_scale, workspace, ws_bytes, stream=None):
    _check("nvfp4_quantize_2d", lib().nvfp4_quantize_2d(
        _p(w), rows, cols, ld, _p(codes_row), _p(codes_col), _p(scales), _p(scales_mma_row), _p(scales_mma_col),
        _p(global_scale), _p(workspace), ws_bytes, _stream(stream)))


def nvfp4_dequantize(codes, scales, scale_mode, global_scale, rows, cols, out_dtype, out, stream=None):
    _check("nvfp4_dequantize", lib().nvfp4_dequantize(
        _p(codes), _p(scales), scale_mode, _p(global_scale), rows, cols, out_dtype, _p(out), _stream(stream)))


def nvfp4_gemm(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, out_dtype, c, ldc,
               stream=None):
    _check("nvfp4_gemm", lib().nvfp4_gemm(
        _p(a_codes), _p(a_scales_mma), _p(a_gs), _p(b_codes), _p(b_scales_mma), _p(b_gs), M, N, K, out_dtype,
        _p(c), ldc, _stream(stream)))


def nvfp4_gemm_amax(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, out_dtype, c, ldc, c_amax,
                    stream=None):
    _check("nvfp4_gemm_amax", lib().nvfp4_gemm_amax(
        _p(a_codes), _p(a_scales_mma), _p(a_gs), _p(b_codes), _p(b_scales_mma), _p(b_gs), M, N, K, out_dtype,
        _p(c), ldc, _p(c_amax), _stream(stream)))


def nvfp4_quantize_1d_from_amax(x, rows, cols, ld, transpose, rounding, sr_seed, amax, codes, scales, scales_mma,
                                global_scale, stream=None):
    _check("nvfp4_quantize_1d_from_amax", lib().nvfp4_quantize_1d_from_amax(
        _p(x), rows, cols, ld, transpose, rounding, sr_seed, _p(amax), _p(codes), _p(scales), _p(scales_mma),
        _p(global_scale), _stream(stream)))


def nvfp4_quantize_2d_from_amax(w, rows, cols, ld, amax, codes_row, codes_col, scales, scales_mma_row,
                                scales_mma_col, global_scale, stream=None):
    _check("nvfp4_quantize_2d_from_amax", lib().nvfp4_quantize_2d_from_amax(
        _p(w), rows, cols, ld, _p(amax), _p(codes_row), _p(codes_col), _p(scales), _p(scales_mma_row),
        _p(scales_mma_col), _p(global_scale), _stream(stream)))


def nvfp4_mxfp4_quantize(x, rows, cols, ld, codes, scales, scales_mma, stream=None):
    _check("nvfp4_mxfp4_quantize", lib().nvfp4_mxfp4_quantize(
        _p(x), rows, cols, ld, _p(codes), _p(scales), _p(scales_mma), _stream(stream)))


def nvfp4_mxfp4_dequantize(codes, scales, rows, cols, out_dtype, out, stream=None):
    _check("nvfp4_mxfp4_dequantize", lib().nvfp4_mxfp4_dequantize(
        _p(codes), _p(scales), rows, cols, out_dtype, _p(out), _stream(stream)))


def nvfp4_mxfp4_gemm(a_codes, a_scales_mma, b_codes, b_scales_mma, M, N, K, out_dtype, c, ldc, stream=None):
    _check("nvfp4_mxfp4_gemm", lib().nvfp4_mxfp4_gemm(
        _p(a_codes), _p(a_scales_mma), _p(b_codes), _p(b_scales_mma), M, N, K, out_dtype, _p(c), ldc,
        _stream(stream)))


def nvfp4_scales_to_mma(scales, scale_mode, rows, k, scales_mma, stream=None):
    _check("nvfp4_scales_to_mma", lib().nvfp4_scales_to_mma(
        _p(scales), scale_mode, rows, k, _p(scales_mma), _stream(stream)))


def nvfp4_gemm_epilogue(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, bias, activation, residual,
                        ldr, out_dtype, c, ldc, pre, ldp, c_amax, stream=None):
    _check("nvfp4_gemm_epilogue", lib().nvfp4_gemm_epilogue(
        _p(a_codes), _p(a_scales_mma), _p(a_gs), _p(b_codes), _p(b_scales_mma), _p(b_gs), M, N, K, _p(bias),
        activation, _p(residual), ldr, out_dtype, _p(c), ldc, _p(pre), ldp, _p(c_amax), _stream(stream)))


def nvfp4_act_grad_workspace_size(M: int, N: int) -> int:
    return lib().nvfp4_act_grad_workspace_size(M, N)


def nvfp4_act_grad(dy, ldy, z, ldz, M, N, activation, offsets, counts, experts, dz, lddz, dbias, amax, workspace,
                   ws_bytes, stream=None):
    _check("nvfp4_act_grad", lib().nvfp4_act_grad(
        _p(dy), ldy, _p(z), ldz, M, N, activation, _p(offsets), _p(counts), experts, _p(dz), lddz, _p(dbias),
        _p(amax), _p(workspace), ws_bytes, _stream(stream)))


def nvfp4_moe_rows(copies: int, experts: int) -> int:
    return lib().nvfp4_moe_rows(copies, experts)


def nvfp4_moe_workspace_size(copies: int, experts: int) -> int:
    return lib().nvfp4_moe_workspace_size(copies, experts)


def nvfp4_moe_sort(expert_ids, copies, experts, rows, offsets, counts, row_copy, copy_row, workspace, ws_bytes,
                   stream=None):
    _check("nvfp4_moe_sort", lib().nvfp4_moe_sort(
        _p(expert_ids), copies, experts, rows, _p(offsets), _p(counts), _p(row_copy), _p(copy_row), _p(workspace),
        ws_bytes, _stream(stream)))


def nvfp4_moe_gather(x, ldx, tokens, topk, cols, copy_row, row_copy, rows, y, ldy, amax, stream=None):
    _check("nvfp4_moe_gather", lib().nvfp4_moe_gather(
        _p(x), ldx, tokens, topk, cols, _p(copy_row), _p(row_copy), rows, _p(y), ldy, _p(amax), _stream(stream)))


def nvfp4_moe_combine(y, ldy, rows, cols, copy_row, weights, residual, ldr, tokens, topk, out, ldo, stream=None):
    _check("nvfp4_moe_combine", lib().nvfp4_moe_combine(
        _p(y), ldy, rows, cols, _p(copy_row), _p(weights), _p(residual), ldr, tokens, topk, _p(out), ldo,
        _stream(stream)))


def nvfp4_moe_combine_grad(dout, ldo, y, ldy, tokens, topk, cols, copy_row, row_copy, rows, weights, dy, lddy,
                           dweights, amax, stream=None):
    _check("nvfp4_moe_combine_grad", lib().nvfp4_moe_combine_grad(
        _p(dout), ldo, _p(y), ldy, tokens, topk, cols, _p(copy_row), _p(row_copy), rows, _p(weights), _p(dy), lddy,
        _p(dweights), _p(amax), _stream(stream)))


def nvfp4_gemm_grouped(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, offsets, counts, experts, M, N, K,
                       bias, activation, residual, ldr, out_dtype, c, ldc, pre, ldp, c_amax, stream=None):
    _check("nvfp4_gemm_grouped", lib().nvfp4_gemm_grouped(
        _p(a_codes), _p(a_scales_mma), _p(a_gs), _p(b_codes), _p(b_scales_mma), _p(b_gs), _p(offsets), _p(counts),
        experts, M, N, K, _p(bias), activation, _p(residual), ldr, out_dtype, _p(c), ldc, _p(pre), ldp, _p(c_amax),
        _stream(stream)))


def nvfp4_gemm_grouped_wgrad(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, offsets, counts, experts, M,
                             N, K, out_dtype, c, ldc, stream=None):
    _check("nvfp4_gemm_grouped_wgrad", lib().nvfp4_gemm_grouped_wgrad(
        _p(a_codes), _p(a_scales_mma), _p(a_gs), _p(b_codes), _p(b_scales_mma), _p(b_gs), _p(offsets), _p(counts),
        experts, M, N, K, out_dtype, _p(c), ldc, _stream(stream)))


def nvfp4_get_error(stream=None) -> int:
    return lib().nvfp4_get_error(_stream(stream))


def nvfp4_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return lib().nvfp4_selftest_wait_timeout(int(limit_ns), _stream(stream))


# --------------------------------------------------------- torch helpers ----
def _tensors(*values):
    """The tensors among values, those in a Quantized, a MoePlan or a tuple included."""
    for v in values:
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, tuple):
            yield from _tensors(*v)
        elif isinstance(v, (Quantized, MoePlan)):
            yield from _tensors(*vars(v).values())


def _torch_stream(stream):
    if not isinstance(stream, int):
        return stream
    # 0 and 1 are the default stream's handles
    return torch.cuda.ExternalStream(stream) if stream > 1 else torch.cuda.default_stream()


def _on_stream(helper):
    """A helper whose `stream` is made the current one while it runs, so that what it allocates belongs to the stream
    that works on it.  The results are used by the caller's stream as well, and the arguments by `stream`: neither
    goes back to the allocator before both are past them."""
    at = list(inspect.signature(helper).parameters).index("stream")

    @functools.wraps(helper)
    def call(*args, **kw):
        stream = kw.get("stream") if len(args) <= at else args[at]
        if stream is None:
            return helper(*args, **kw)
        here, there = torch.cuda.current_stream(), _torch_stream(stream)
        with torch.cuda.stream(there):
            result = helper(*args, **kw)
        if here.cuda_stream != there.cuda_stream:
            for t in _tensors(*args, *kw.values()):
                t.record_stream(there)
            for t in _tensors(result):
                t.record_stream(here)
        return result
    return call


@dataclass
class Quantized:
    """One NVFP4 tensor Q [rows x cols] on the device."""
    codes: torch.Tensor                      # uint8 [rows, cols/2]
    scales: Optional[torch.Tensor]           # uint8 plain layout
    scales_mma: Optional[torch.Tensor]       # uint8 MMA layout
    global_scale: torch.Tensor               # float32 [1]
    rows: int
    cols: int
    codes_col: Optional[torch.Tensor] = None         # 2D only: codes of Q^T
    scales_mma_col: Optional[torch.Tensor] = None    # 2D only: MMA scales of Q^T


_ws_cache = {}


def workspace(device=None) -> torch.Tensor:
    """A per-device scratch buffer for the amax partials (allocated by torch), for callers of the C names that use one
    stream at a time; the helpers take scratch of their own in each call."""
    dev = torch.device(device if device is not None else "cuda")
    key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device())
    ws = _ws_cache.get(key)
    n = nvfp4_workspace_size(0, 0)
    if ws is None or ws.numel() < n:
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        _ws_cache[key] = ws
    return ws


def _scratch(nbytes: int, device) -> torch.Tensor:
    """Device scratch of one call, allocated on the stream that it is used on."""
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def _empty_u8(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device)


@_on_stream
def quantize_1d(x: torch.Tensor, transpose: bool = False, rounding: int = NVFP4_RNE, sr_seed: int = 0,
                rht: bool = False, rht_seed: int = 0, plain_scales: bool = True, mma_scales: bool = True,
                stream=None, amax: Optional[torch.Tensor] = None, rht_order: int = 16) -> Quantized:
    """Quantize a bf16 [rows x cols] tensor (or its transpose) with 16-element blocks.
    With `amax` (a device float holding max |x|) the amax pass is skipped;
    with `rht` the Q rows are rotated in chunks of `rht_order` points."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    qr, qc = (cols, rows) if transpose else (rows, cols)
    dev = x.device
    codes = torch.empty(qr, qc // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(qr, qc // 16, dtype=torch.uint8, device=dev) if plain_scales else None
    smma = _empty_u8(nvfp4_mma_scale_bytes(qr, qc), dev) if mma_scales else None
    gs = torch.empty(1, dtype=torch.float32, device=dev)
    ws = _scratch(nvfp4_workspace_size(rows, cols), dev) if amax is None else None
    if amax is not None:
        assert not rht, "the amax of the rotated tensor is not known to a producer"
        nvfp4_quantize_1d_from_amax(x, rows, cols, x.stride(0), int(transpose), rounding, sr_seed, amax, codes,
                                    scales, smma, gs, stream)
    elif rht and rht_order != 16:
        nvfp4_rht_quantize_n(x, rows, cols, x.stride(0), int(transpose), rht_order, rht_seed, rounding, sr_seed,
                             codes, scales, smma, gs, ws, ws.numel(), stream)
    elif rht:
        nvfp4_rht_quantize_sr(x, rows, cols, x.stride(0), int(transpose), rht_seed, rounding, sr_seed, codes,
                              scales, smma, gs, ws, ws.numel(), stream)
    else:
        nvfp4_quantize_1d(x, rows, cols, x.stride(0), int(transpose), rounding, sr_seed, codes, scales, smma,
                          gs, ws, ws.numel(), stream)
    return Quantized(codes, scales, smma, gs, qr, qc)


@_on_stream
def quantize_2d(w: torch.Tensor, columnwise: bool = True, plain_scales: bool = True, mma_scales: bool = True,
                stream=None, amax: Optional[torch.Tensor] = None) -> Quantized:
    """Quantize a bf16 weight with 16x16 tiles (rowwise codes, optional columnwise copy)."""
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    rows, cols = w.shape
    dev = w.device
    cr = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    cc = torch.empty(cols, rows // 2, dtype=torch.uint8, device=dev) if columnwise else None
    sc = torch.empty(rows // 16, cols // 16, dtype=torch.uint8, device=dev) if plain_scales else None
    mr = _empty_u8(nvfp4_mma_scale_bytes(rows, cols), dev) if mma_scales else None
    mc = _empty_u8(nvfp4_mma_scale_bytes(cols, rows), dev) if (mma_scales and columnwise) else None
    gs = torch.empty(1, dtype=torch.float32, device=dev)
    ws = _scratch(nvfp4_workspace_size(rows, cols), dev) if amax is None else None
    if amax is not None:
        nvfp4_quantize_2d_from_amax(w, rows, cols, w.stride(0), amax, cr, cc, sc, mr, mc, gs, stream)
    else:
        nvfp4_quantize_2d(w, rows, cols, w.stride(0), cr, cc, sc, mr, mc, gs, ws, ws.numel(), stream)
    return Quantized(cr, sc, mr, gs, rows, cols, codes_col=cc, scales_mma_col=mc)


@_on_stream
def dequantize(q: Quantized, scale_mode: int = NVFP4_SCALE_1D, out_dtype: int = NVFP4_OUT_F32,
               stream=None) -> torch.Tensor:
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    out = torch.empty(q.rows, q.cols, dtype=dt, device=q.codes.device)
    nvfp4_dequantize(q.codes, q.scales, scale_mode, q.global_scale, q.rows, q.cols, out_dtype, out, stream)
    return out


@_on_stream
def gemm(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M: int, N: int, K: int,
         out_dtype: int = NVFP4_OUT_BF16, out: Optional[torch.Tensor] = None, stream=None,
         amax_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = alpha * A . B^T with NVFP4 operands (MMA-layout scales).  With
    `amax_out` (a device float) the epilogue also writes max |C| there."""
    if out is None:
        dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
        ldc = (N + 7) // 8 * 8
        out = torch.empty(M, ldc, dtype=dt, device=a_codes.device)[:, :N]
    if amax_out is not None:
        nvfp4_gemm_amax(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, out_dtype, out,
                        out.stride(0), amax_out, stream)
    else:
        nvfp4_gemm(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, out_dtype, out,
                   out.stride(0), stream)
    return out


@_on_stream
def mxfp4_quantize(x: torch.Tensor, plain_scales: bool = True, mma_scales: bool = True, stream=None) -> Quantized:
    """MXFP4 quantization of a bf16 [rows x cols] tensor (32-element blocks, E8M0 scales)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    dev = x.device
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=dev) if plain_scales else None
    smma = _empty_u8(nvfp4_mma_scale_bytes(rows, cols), dev) if mma_scales else None
    nvfp4_mxfp4_quantize(x, rows, cols, x.stride(0), codes, scales, smma, stream)
    return Quantized(codes, scales, smma, torch.ones(1, dtype=torch.float32, device=dev), rows, cols)


@_on_stream
def mxfp4_gemm(a: Quantized, b: Quantized, out_dtype: int = NVFP4_OUT_BF16, stream=None) -> torch.Tensor:
    """C = A . B^T of two MXFP4 operands (K-major)."""
    M, K, N = a.rows, a.cols, b.rows
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    ldc = (N + 7) // 8 * 8
    out = torch.empty(M, ldc, dtype=dt, device=a.codes.device)[:, :N]
    nvfp4_mxfp4_gemm(a.codes, a.scales_mma, b.codes, b.scales_mma, M, N, K, out_dtype, out, out.stride(0), stream)
    return out


@_on_stream
def quantize_dual(x: torch.Tensor, rounding: int = NVFP4_RNE, sr_seed: int = 0, rht_seed: int = 0,
                  sr_seed_t: int = 0, stream=None):
    """(Q1, Q2): x row-wise and RHT(x^T), from one shared amax read."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    dev = x.device
    q1 = Quantized(torch.empty(rows, cols // 2, dtype=torch.uint8, device=dev),
                   torch.empty(rows, cols // 16, dtype=torch.uint8, device=dev),
                   _empty_u8(nvfp4_mma_scale_bytes(rows, cols), dev), torch.empty(1, dtype=torch.float32, device=dev),
                   rows, cols)
    q2 = Quantized(torch.empty(cols, rows // 2, dtype=torch.uint8, device=dev),
                   torch.empty(cols, rows // 16, dtype=torch.uint8, device=dev),
                   _empty_u8(nvfp4_mma_scale_bytes(cols, rows), dev), torch.empty(1, dtype=torch.float32, device=dev),
                   cols, rows)
    ws = torch.empty(2 * nvfp4_workspace_size(rows, cols), dtype=torch.uint8, device=dev)
    nvfp4_quantize_dual(x, rows, cols, x.stride(0), rounding, sr_seed, q1.codes, q1.scales, q1.scales_mma,
                        q1.global_scale, rht_seed, sr_seed_t, q2.codes, q2.scales, q2.scales_mma, q2.global_scale,
                        ws, ws.numel(), stream)
    return q1, q2


# ------------------------------------------------------ the linear layer ----
def _here(*tensors: torch.Tensor):
    """Launches go to the current device: a tensor elsewhere (host memory included) is refused."""
    dev = _current_device()
    for t in tensors:
        assert t.get_device() == dev, f"tensor on {t.device}, not on the current CUDA device"


def _matrix(t: torch.Tensor, rows: int, cols: int, dtype=torch.bfloat16) -> int:
    """Row stride of a [rows x cols] matrix with unit column stride (checked)."""
    assert t.dtype is dtype and t.shape == (rows, cols)
    _here(t)
    ld, unit = t.stride()
    assert unit == 1 or cols == 1
    return ld if rows > 1 else (cols + 7) // 8 * 8


def _padded(rows: int, cols: int, dtype, like: torch.Tensor) -> torch.Tensor:
    """A [rows x cols] view, on the device of `like`, whose row stride is a multiple of 8 elements."""
    ld = (cols + 7) // 8 * 8
    t = like.new_empty((rows, ld), dtype=dtype)
    return t if ld == cols else t.narrow(1, 0, cols)


def _check_operand(codes, scales_mma, gs, rows: int, k: int, experts: int = 1):
    assert codes.dtype is torch.uint8 and codes.numel() == experts * rows * (k // 2) and codes.is_contiguous()
    need = (rows + 127) // 128 * ((k // 16 + 3) // 4) * 512      # nvfp4_mma_scale_bytes
    assert scales_mma.element_size() == 1 and scales_mma.numel() >= experts * need and scales_mma.is_contiguous()
    assert gs.dtype is torch.float32 and gs.numel() == experts and gs.is_contiguous()
    _here(codes, scales_mma, gs)


def _check_word(t):
    if t is not None:
        assert t.dtype is torch.float32 and t.numel() == 1
        _here(t)


@_on_stream
def gemm_epilogue(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M: int, N: int, K: int, bias=None,
                  activation: int = NVFP4_ACT_NONE, residual: Optional[torch.Tensor] = None,
                  out_dtype: int = NVFP4_OUT_BF16, out: Optional[torch.Tensor] = None,
                  pre: Optional[torch.Tensor] = None, amax_out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """C = act(alpha * A . B^T + bias) + residual with NVFP4 operands (MMA-layout scales).

    bias bf16 [N]; residual bf16 [M x N], which may be `out`; `pre` (bf16 [M x N]) receives the
    pre-activation and `amax_out` (a device float) max |C|."""
    _check_operand(a_codes, a_scales_mma, a_gs, M, K)
    _check_operand(b_codes, b_scales_mma, b_gs, N, K)
    return _gemm_layer(None, a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, bias, activation,
                       residual, out_dtype, out, pre, amax_out, stream)


def _gemm_layer(plan, a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, bias, activation, residual,
                out_dtype, out, pre, amax_out, stream):
    experts = 1 if plan is None else plan.experts
    if bias is not None:
        assert bias.dtype is torch.bfloat16 and bias.is_contiguous() and bias.numel() == experts * N
        _here(bias)
    _check_word(amax_out)
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = _padded(M, N, dt, a_codes)
    ldc = _matrix(out, M, N, dt)
    ldr = _matrix(residual, M, N) if residual is not None else 0
    ldp = _matrix(pre, M, N) if pre is not None else 0
    if plan is None:
        nvfp4_gemm_epilogue(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, bias, activation,
                            residual, ldr, out_dtype, out, ldc, pre, ldp, amax_out, stream)
    else:
        nvfp4_gemm_grouped(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, plan.offsets, plan.counts,
                           experts, M, N, K, bias, activation, residual, ldr, out_dtype, out, ldc, pre, ldp,
                           amax_out, stream)
    return out


@_on_stream
def act_grad(dy: torch.Tensor, z: Optional[torch.Tensor], activation: int, bias_grad: bool = True,
             plan: "Optional[MoePlan]" = None, out: Optional[torch.Tensor] = None,
             amax_out: Optional[torch.Tensor] = None, stream=None):
    """(dz, dbias) of C = act(z) + residual with z = product + bias: dz = dy * act'(z) in bf16, dbias its column
    sums in fp32 ([N], with a plan [experts x N]; None without bias_grad).  z is the `pre` of gemm_epilogue."""
    M, N = dy.shape
    if plan is not None:
        assert plan.rows == M
        _here(plan.counts)
    ldy = _matrix(dy, M, N)
    ldz = _matrix(z, M, N) if z is not None else 0
    if out is None:
        out = _padded(M, N, torch.bfloat16, dy)
    lddz = _matrix(out, M, N)
    _check_word(amax_out)
    dbias = ws = None
    experts = 0 if plan is None else plan.experts
    if bias_grad:
        dbias = dy.new_empty((experts, N) if experts else (N,), dtype=torch.float32)
        ws = _scratch(nvfp4_act_grad_workspace_size(M, N), dy.device)
    nvfp4_act_grad(dy, ldy, z, ldz, M, N, activation, plan.offsets if experts else None,
                   plan.counts if experts else None, experts, out, lddz, dbias, amax_out, ws,
                   ws.numel() if bias_grad else 0, stream)
    return out, dbias


# --------------------------------------------------- the layer of experts ---
@dataclass
class MoePlan:
    """Where the copies of routed tokens go: rows sorted by expert (int32 device tensors, see nvfp4_moe_sort)."""
    offsets: torch.Tensor    # [experts + 1]
    counts: torch.Tensor     # [experts]
    row_copy: torch.Tensor   # [rows]
    copy_row: torch.Tensor   # [tokens, topk]

    def __post_init__(self):
        for t in (self.offsets, self.counts, self.row_copy, self.copy_row):
            assert t.dtype is torch.int32 and t.is_contiguous() and t.device == self.copy_row.device
        self.experts = self.counts.numel()
        self.rows = self.row_copy.numel()
        assert self.offsets.numel() == self.experts + 1
        self.tokens, self.topk = self.copy_row.shape


@_on_stream
def moe_sort(expert_ids: torch.Tensor, experts: int, rows: Optional[int] = None, stream=None) -> MoePlan:
    """Sort the copies of int32 expert_ids [tokens x topk] by expert.  rows (default: enough for every routing)
    bounds the sorted matrices; copies that find no row are dropped."""
    assert expert_ids.dtype is torch.int32 and expert_ids.dim() == 2 and expert_ids.is_contiguous()
    _here(expert_ids)
    n = expert_ids.numel()
    if rows is None:
        rows = (n + 127 * min(n, experts) + 127) // 128 * 128        # nvfp4_moe_rows
    ws_bytes = nvfp4_moe_workspace_size(n, experts)
    # one allocation: the call's scratch, then the plan's four arrays
    sizes = (ws_bytes // 4, experts + 1, experts, rows, n)
    buf = expert_ids.new_empty(sum(sizes))
    ws = buf.data_ptr()
    offsets = ws + ws_bytes
    counts = offsets + 4 * experts + 4
    row_copy = counts + 4 * experts
    nvfp4_moe_sort(expert_ids, n, experts, rows, offsets, counts, row_copy, row_copy + 4 * rows, ws, ws_bytes, stream)
    _, offsets, counts, row_copy, copy_row = torch.split_with_sizes(buf, sizes)
    return MoePlan(offsets, counts, row_copy, copy_row.view(expert_ids.shape))


@_on_stream
def moe_gather(x: torch.Tensor, plan: MoePlan, out: Optional[torch.Tensor] = None,
               amax_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The token rows x bf16 [tokens x cols] sorted by expert: bf16 [rows x cols], zeros in padding rows.  With
    `amax_out` (a device float) also max |x|, for the quantizers.  Its gradient is moe_combine without weights."""
    cols = x.shape[1]
    _here(plan.copy_row)
    if out is None:
        out = x.new_empty((plan.rows, cols))
    _check_word(amax_out)
    nvfp4_moe_gather(x, _matrix(x, plan.tokens, cols), plan.tokens, plan.topk, cols, plan.copy_row, plan.row_copy,
                     plan.rows, out, _matrix(out, plan.rows, cols), amax_out, stream)
    return out


def _check_weights(weights, plan):
    if weights is not None:
        assert weights.dtype is torch.float32 and weights.is_contiguous() and weights.shape == plan.copy_row.shape
        _here(weights)


@_on_stream
def moe_combine(y: torch.Tensor, plan: MoePlan, weights: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """residual[t] + sum_j weights[t, j] * y[row of copy (t, j)]: bf16 [tokens x cols]; weights fp32 or None (1)."""
    cols = y.shape[1]
    _here(plan.copy_row)
    _check_weights(weights, plan)
    if out is None:
        out = y.new_empty((plan.tokens, cols))
    nvfp4_moe_combine(y, _matrix(y, plan.rows, cols), plan.rows, cols, plan.copy_row, weights, residual,
                      _matrix(residual, plan.tokens, cols) if residual is not None else 0, plan.tokens, plan.topk,
                      out, _matrix(out, plan.tokens, cols), stream)
    return out


@_on_stream
def moe_combine_grad(dout: torch.Tensor, y: Optional[torch.Tensor], plan: MoePlan,
                     weights: Optional[torch.Tensor] = None, amax_out: Optional[torch.Tensor] = None, stream=None):
    """(dy, dweights) of moe_combine: dy bf16 [rows x cols] with zeros in padding rows, dweights fp32
    [tokens x topk] (None when y is None)."""
    cols = dout.shape[1]
    _here(plan.copy_row)
    _check_weights(weights, plan)
    _check_word(amax_out)
    dy = dout.new_empty((plan.rows, cols))
    dw = dout.new_empty(plan.copy_row.shape, dtype=torch.float32) if y is not None else None
    nvfp4_moe_combine_grad(dout, _matrix(dout, plan.tokens, cols), y,
                           _matrix(y, plan.rows, cols) if y is not None else 0, plan.tokens, plan.topk, cols,
                           plan.copy_row, plan.row_copy, plan.rows, weights, dy, cols, dw, amax_out, stream)
    return dy, dw


@_on_stream
def gemm_grouped(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, plan: MoePlan, M: int, N: int, K: int,
                 bias=None, activation: int = NVFP4_ACT_NONE, residual: Optional[torch.Tensor] = None,
                 out_dtype: int = NVFP4_OUT_BF16, out: Optional[torch.Tensor] = None,
                 pre: Optional[torch.Tensor] = None, amax_out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """gemm_epilogue over M rows sorted by expert: b_codes [experts x N x K/2], their scales and b_gs [experts],
    bias [experts x N].  Padding rows of C (and pre) are zeros."""
    assert plan.rows == M
    _here(plan.counts)
    _check_operand(a_codes, a_scales_mma, a_gs, M, K)
    _check_operand(b_codes, b_scales_mma, b_gs, N, K, plan.experts)
    return _gemm_layer(plan, a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, M, N, K, bias, activation,
                       residual, out_dtype, out, pre, amax_out, stream)


@_on_stream
def gemm_grouped_wgrad(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, plan: MoePlan, M: int, N: int,
                       K: int, out_dtype: int = NVFP4_OUT_F32, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """[experts x M x N]: per expert A . B^T over its K sorted rows, A [M x K] and B [N x K] the transposed
    operands."""
    assert plan.rows == K
    _here(plan.counts)
    _check_operand(a_codes, a_scales_mma, a_gs, M, K)
    _check_operand(b_codes, b_scales_mma, b_gs, N, K)
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = _padded(plan.experts * M, N, dt, a_codes).unflatten(0, (plan.experts, M))
    assert out.dtype is dt and out.shape == (plan.experts, M, N) and out.stride(2) == 1
    _here(out)
    assert plan.experts == 1 or out.stride(0) == M * out.stride(1)
    nvfp4_gemm_grouped_wgrad(a_codes, a_scales_mma, a_gs, b_codes, b_scales_mma, b_gs, plan.offsets, plan.counts,
                             plan.experts, M, N, K, out_dtype, out, out.stride(1), stream)
    return out


@_on_stream
def quantize_2d_experts(w: torch.Tensor, columnwise: bool = True, stream=None):
    """(W, W^T) operands of gemm_grouped from expert weights bf16 [experts x rows x cols], each quantized by
    quantize_2d: Quantized with stacked codes, scales and global scales (the second None without columnwise)."""
    assert w.dtype is torch.bfloat16 and w.dim() == 3 and w.stride(2) == 1
    _here(w)
    experts, rows, cols = w.shape
    dev = w.device
    row = Quantized(torch.empty(experts, rows, cols // 2, dtype=torch.uint8, device=dev), None,
                    torch.empty(experts, nvfp4_mma_scale_bytes(rows, cols), dtype=torch.uint8, device=dev),
                    torch.empty(experts, dtype=torch.float32, device=dev), rows, cols)
    col = Quantized(torch.empty(experts, cols, rows // 2, dtype=torch.uint8, device=dev), None,
                    torch.empty(experts, nvfp4_mma_scale_bytes(cols, rows), dtype=torch.uint8, device=dev),
                    row.global_scale, cols, rows) if columnwise else None
    ws = _scratch(nvfp4_workspace_size(rows, cols), dev)
    for e in range(experts):
        nvfp4_quantize_2d(w[e], rows, cols, w.stride(1), row.codes[e], col.codes[e] if columnwise else None, None,
                          row.scales_mma[e], col.scales_mma[e] if columnwise else None, row.global_scale[e:e + 1],
                          ws, ws.numel(), stream)
    return row, col
