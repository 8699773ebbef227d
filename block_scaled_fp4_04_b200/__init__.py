"""Python binding of libfp4 (block-scaled FP4 quantization and GEMM for B200).

Argument marshalling only: every step of the quantize / GEMM path runs in the CUDA
kernels of ``libfp4.so`` (built from ``csrc/`` by ``build.py``).  PyTorch provides
device memory and streams.  There is no CPU fallback: if the shared library is
missing or the device is not an sm_100 GPU, the calls raise.

The functions named ``fp4_*`` mirror the C entry points of ``include/fp4.h`` one to
one (tensors stand in for device pointers).  ``quantize``, ``gemm`` and the functions
after them are conveniences that allocate the outputs with torch and call them.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4.so")

NVFP4, MXFP4, MXFP8 = 0, 1, 2  # MXFP8: E4M3 elements, one byte each (the mixed GEMM's FP8 operand)
F32, BF16 = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_NONFINITE = range(6)
GEMM_WEIGHTS_READY = 1
QUANT_E8M0_FLOOR = 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)
_STATUS_NAMES = {0: "FP4_OK", 1: "FP4_ERR_INVALID_ARG", 2: "FP4_ERR_UNSUPPORTED", 3: "FP4_ERR_CUDA",
                 4: "FP4_ERR_TIMEOUT", 5: "FP4_ERR_NONFINITE"}

_lib = None
_lock = threading.Lock()


class Fp4Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libfp4.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m block_scaled_fp4_04_b200.build` (no CPU fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            sigs = {
                "fp4_version": (ctypes.c_char_p, []),
                "fp4_last_error": (ctypes.c_char_p, []),
                "fp4_scales_bytes": (SZ, [I64, I64, I32]),
                "fp4_scales_bytes_grouped": (SZ, [I64, I32, I64, I32]),
                "fp4_quantize_workspace_size": (SZ, []),
                "fp4_amax": (I32, [P, I64, I32, P, P, SZ, P]),
                "fp4_quantize": (I32, [P, I64, I64, I32, I32, I32, P, P, P, P, P, P, P, SZ, P]),
                "fp4_quantize_grouped": (I32, [P, I64, I64, I32, I32, I32, P, P, P, P, P, P, SZ, P]),
                "fp4_quantize_ex": (I32, [P, I64, I64, I32, I32, I32, ctypes.c_uint, P, P, P, P, P, P, P, SZ, P]),
                "fp4_quantize_sr": (I32, [P, I64, I64, I32, P, P, P, P, P, P, SZ, P]),
                "fp4_quantize_rht": (I32, [P, I64, I64, I32, I32, ctypes.c_uint32, P, P, P, P, P, SZ, P]),
                "fp4_global_scale": (I32, [P, P, P]),
                "fp4_dequantize": (I32, [P, P, P, I64, I64, I32, P, P]),
                "fp4_gemm_workspace_size": (SZ, [I64, I64, I64, I32]),
                "fp4_gemm": (I32, [I32, P, P, P, P, P, P, I64, I64, I64, P, I32, P, SZ, P]),
                "fp4_gemm_ex": (I32, [I32, P, P, P, P, P, P, I64, I64, I64, P, I32, P, SZ, ctypes.c_uint, P]),
                "fp4_gemm_noalloc": (I32, [I32, P, P, P, P, P, P, I64, I64, I64, P, I32, P]),
                "fp4_gemm_mixed": (I32, [I32, P, P, I32, P, P, I64, I64, I64, P, I32, P]),
                "fp4_gemm_epilogue_workspace_size": (SZ, [I64, I64, I64, I32, I32]),
                "fp4_gemm_epilogue": (I32, [I32, P, P, P, P, P, P, I64, I64, I64, P, I32, P, I32, P, P, P, P, P,
                                            SZ, P]),
                "fp4_gemm_bf16a_workspace_size": (SZ, [I64, I64, I64]),
                "fp4_gemm_bf16a": (I32, [P, P, P, P, I64, I64, I64, P, I32, P, P, P, P, SZ, ctypes.c_uint, P]),
                "fp4_gemm_grouped": (I32, [I32, I32, P, P, P, P, P, P, P, I64, I64, I64, P, I32, P, SZ, P]),
                "fp4_gemm_epilogue_ex": (I32, [I32, P, P, P, P, P, P, I64, I64, I64, P, I32, P, I32, P, I32, P, P, P, P,
                                               P, P, SZ, ctypes.c_uint, P]),
                "fp4_gemm_gated_workspace_size": (SZ, [I64, I64, I64, I32, I32]),
                "fp4_gemm_gated": (I32, [I32, P, P, P, P, P, P, P, P, P, I64, I64, I64, P, P, I32, P, I32, P, P, P, P, P,
                                         P, P, SZ, ctypes.c_uint, P]),
                "fp4_gemm_gated_bf16a_workspace_size": (SZ, [I64, I64, I64]),
                "fp4_gemm_gated_bf16a": (I32, [P, P, P, P, P, P, P, I64, I64, I64, P, P, I32, P, I32, P, P, P, P, P, P,
                                               SZ, ctypes.c_uint, P]),
                "fp4_gemm_gated_grouped": (I32, [I32, I32, P, P, P, P, P, P, P, P, P, P, I64, I64, I64, P, P, I32, P,
                                                 I32, P, P, P]),
                "fp4_act_backward_workspace_size": (SZ, [I64, I64, I32]),
                "fp4_act_backward": (I32, [P, P, P, I64, I64, I32, I32, P, I32, P, I32, P, P, P, P, P, SZ, P]),
                "fp4_layernorm": (I32, [P, I64, I64, I32, P, P, ctypes.c_float, P, I32, P, P, I32, P, P, P, P, P]),
                "fp4_layernorm_backward_workspace_size": (SZ, [I64, I64]),
                "fp4_layernorm_backward": (I32, [P, P, I64, I64, I32, P, P, P, P, P, I32, P, P, P, SZ, P]),
                "fp4_moe_sort_workspace_size": (SZ, [I64, I32, I32]),
                "fp4_moe_sort": (I32, [P, I32, I64, I32, I32, P, P, P, P, SZ, P]),
                "fp4_moe_dispatch": (I32, [P, I64, I64, I32, I32, P, P, I32, P]),
                "fp4_moe_dispatch_codes": (I32, [P, I64, I64, I32, I32, P, P, I32, P, I32, P, P, P, P]),
                "fp4_moe_dispatch_i8": (I32, [P, I64, I64, I32, I32, P, P, P, P]),
                "fp4_moe_combine": (I32, [P, I32, P, P, I64, I32, I64, P, I32, P, I32, P]),
                "fp4_moe_combine_backward": (I32, [P, P, I32, P, P, I64, I32, I64, P, I32, P, P]),
                "fp4_quantize_i8": (I32, [P, I64, I64, I32, P, P, P, P]),
                "fp4_gemm_i8_workspace_size": (SZ, [I64, I64, I64]),
                "fp4_gemm_i8": (I32, [P, P, P, P, I64, I64, I64, P, I32, P, I32, P, SZ, ctypes.c_uint, P]),
                "fp4_gemm_i8_grouped_workspace_size": (SZ, [I32, I64, I64, I64]),
                "fp4_gemm_i8_grouped": (I32, [I32, P, P, P, P, P, I64, I64, I64, P, I32, P, I32, P, SZ, P]),
                "fp4_get_status": (I32, [P]),
                "fp4_debug_encode": (I32, [P, I64, I32, P, P]),
                "fp4_debug_stall_next_decode": (I32, [I32]),
                "fp4_mma_peak": (I32, [I32, I32, P, P]),
            }
            for name, (res, args) in sigs.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _p(t) -> Optional[int]:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != OK:
        raise Fp4Error(rc, lib().fp4_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"input must be float32 or bfloat16, got {t.dtype}")


# ---------------------------------------------------------------- C entry points
def fp4_version() -> str:
    return lib().fp4_version().decode()


def fp4_last_error() -> str:
    return lib().fp4_last_error().decode()


def fp4_scales_bytes(rows: int, cols: int, fmt: int) -> int:
    return int(lib().fp4_scales_bytes(rows, cols, fmt))


def fp4_scales_bytes_grouped(total_rows: int, num_groups: int, cols: int, fmt: int) -> int:
    return int(lib().fp4_scales_bytes_grouped(total_rows, num_groups, cols, fmt))


def fp4_quantize_workspace_size() -> int:
    return int(lib().fp4_quantize_workspace_size())


def fp4_gemm_workspace_size(M: int, N: int, K: int, fmt: int) -> int:
    return int(lib().fp4_gemm_workspace_size(M, N, K, fmt))


def fp4_amax(x, n, in_dtype, amax_out, workspace, workspace_bytes, stream=None):
    _check(lib().fp4_amax(_p(x), n, in_dtype, _p(amax_out), _p(workspace), workspace_bytes, _s(stream)))


def fp4_quantize(x, rows, cols, in_dtype, fmt, block, codes_out, scales_out, global_out,
                 codesT_out=None, scalesT_out=None, global_in=None, workspace=None, workspace_bytes=0,
                 stream=None):
    _check(lib().fp4_quantize(_p(x), rows, cols, in_dtype, fmt, block, _p(codes_out), _p(scales_out),
                              _p(global_out), _p(codesT_out), _p(scalesT_out), _p(global_in), _p(workspace),
                              workspace_bytes, _s(stream)))


def fp4_quantize_grouped(x, rows, cols, in_dtype, fmt, num_groups, offsets, codes_out, scales_out, global_out,
                         global_in=None, workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_quantize_grouped(_p(x), rows, cols, in_dtype, fmt, num_groups, _p(offsets), _p(codes_out),
                                      _p(scales_out), _p(global_out), _p(global_in), _p(workspace),
                                      workspace_bytes, _s(stream)))


def fp4_quantize_ex(x, rows, cols, in_dtype, fmt, block, flags, codes_out, scales_out, global_out,
                    codesT_out=None, scalesT_out=None, global_in=None, workspace=None, workspace_bytes=0,
                    stream=None):
    _check(lib().fp4_quantize_ex(_p(x), rows, cols, in_dtype, fmt, block, flags, _p(codes_out), _p(scales_out),
                                 _p(global_out), _p(codesT_out), _p(scalesT_out), _p(global_in), _p(workspace),
                                 workspace_bytes, _s(stream)))


def fp4_quantize_sr(x, rows, cols, in_dtype, rbits, codes_out, scales_out, global_out, global_in=None,
                    workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_quantize_sr(_p(x), rows, cols, in_dtype, _p(rbits), _p(codes_out), _p(scales_out),
                                 _p(global_out), _p(global_in), _p(workspace), workspace_bytes, _s(stream)))


def fp4_quantize_rht(x, rows, cols, in_dtype, fmt, signs, codes_out, scales_out, global_out, global_in=None,
                     workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_quantize_rht(_p(x), rows, cols, in_dtype, fmt, signs, _p(codes_out), _p(scales_out),
                                  _p(global_out), _p(global_in), _p(workspace), workspace_bytes, _s(stream)))


def fp4_global_scale(amax, global_out, stream=None):
    _check(lib().fp4_global_scale(_p(amax), _p(global_out), _s(stream)))


def fp4_dequantize(codes, scales, global_, rows, cols, fmt, out, stream=None):
    _check(lib().fp4_dequantize(_p(codes), _p(scales), _p(global_), rows, cols, fmt, _p(out), _s(stream)))


def fp4_gemm(fmt, A, sA, gA, B, sB, gB, M, N, K, D, out_dtype, workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_gemm(fmt, _p(A), _p(sA), _p(gA), _p(B), _p(sB), _p(gB), M, N, K, _p(D), out_dtype,
                          _p(workspace), workspace_bytes, _s(stream)))


def fp4_gemm_ex(fmt, A, sA, gA, B, sB, gB, M, N, K, D, out_dtype, workspace=None, workspace_bytes=0, flags=0,
                stream=None):
    _check(lib().fp4_gemm_ex(fmt, _p(A), _p(sA), _p(gA), _p(B), _p(sB), _p(gB), M, N, K, _p(D), out_dtype,
                             _p(workspace), workspace_bytes, flags, _s(stream)))


def fp4_gemm_epilogue_workspace_size(M: int, N: int, K: int, fmt: int, rows_in_place: bool) -> int:
    return int(lib().fp4_gemm_epilogue_workspace_size(M, N, K, fmt, 1 if rows_in_place else 0))


def fp4_gemm_epilogue(fmt, A, sA, gA, B, sB, gB, M, N, K, bias, act, D, out_dtype, Dcodes=None, Dscales=None,
                      gD=None, amax_out=None, workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_gemm_epilogue(fmt, _p(A), _p(sA), _p(gA), _p(B), _p(sB), _p(gB), M, N, K, _p(bias), act, _p(D),
                                   out_dtype, _p(Dcodes), _p(Dscales), _p(gD), _p(amax_out), _p(workspace),
                                   workspace_bytes, _s(stream)))


def fp4_gemm_bf16a_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().fp4_gemm_bf16a_workspace_size(M, N, K))


def fp4_gemm_bf16a(X, B, sB, gB, M, N, K, D, out_dtype, Xcodes, Xscales, gX, workspace, workspace_bytes, flags=0,
                   stream=None):
    _check(lib().fp4_gemm_bf16a(_p(X), _p(B), _p(sB), _p(gB), M, N, K, _p(D), out_dtype, _p(Xcodes), _p(Xscales),
                                _p(gX), _p(workspace), workspace_bytes, flags, _s(stream)))


def fp4_gemm_epilogue_ex(fmt, A, sA, gA, B, sB, gB, M, N, K, bias, act, residual, residual_dtype, D, out_dtype,
                         pre=None, Dcodes=None, Dscales=None, gD=None, amax_out=None, workspace=None,
                         workspace_bytes=0, flags=0, stream=None):
    _check(lib().fp4_gemm_epilogue_ex(fmt, _p(A), _p(sA), _p(gA), _p(B), _p(sB), _p(gB), M, N, K, _p(bias), act,
                                      _p(residual), residual_dtype, _p(D), out_dtype, _p(pre), _p(Dcodes), _p(Dscales),
                                      _p(gD), _p(amax_out), _p(workspace), workspace_bytes, flags, _s(stream)))


def fp4_gemm_gated_workspace_size(M: int, F: int, K: int, fmt: int, rows_in_place: bool) -> int:
    return int(lib().fp4_gemm_gated_workspace_size(M, F, K, fmt, 1 if rows_in_place else 0))


def fp4_gemm_gated(fmt, A, sA, gA, Wg, sWg, gWg, Wu, sWu, gWu, M, F, K, bias_g, bias_u, act, H, out_dtype, G=None,
                   U=None, Hcodes=None, Hscales=None, gH=None, amax_out=None, workspace=None, workspace_bytes=0,
                   flags=0, stream=None):
    _check(lib().fp4_gemm_gated(fmt, _p(A), _p(sA), _p(gA), _p(Wg), _p(sWg), _p(gWg), _p(Wu), _p(sWu), _p(gWu), M, F,
                                K, _p(bias_g), _p(bias_u), act, _p(H), out_dtype, _p(G), _p(U), _p(Hcodes),
                                _p(Hscales), _p(gH), _p(amax_out), _p(workspace), workspace_bytes, flags, _s(stream)))


def fp4_gemm_gated_bf16a_workspace_size(M: int, F: int, K: int) -> int:
    return int(lib().fp4_gemm_gated_bf16a_workspace_size(M, F, K))


def fp4_gemm_gated_bf16a(X, Wg, sWg, gWg, Wu, sWu, gWu, M, F, K, bias_g, bias_u, act, H, out_dtype, G, U, Xcodes,
                         Xscales, gX, workspace, workspace_bytes, flags=0, stream=None):
    _check(lib().fp4_gemm_gated_bf16a(_p(X), _p(Wg), _p(sWg), _p(gWg), _p(Wu), _p(sWu), _p(gWu), M, F, K, _p(bias_g),
                                      _p(bias_u), act, _p(H), out_dtype, _p(G), _p(U), _p(Xcodes), _p(Xscales),
                                      _p(gX), _p(workspace), workspace_bytes, flags, _s(stream)))


def fp4_gemm_gated_grouped(fmt, num_groups, offsets, A, sA, gA, Wg, sWg, gWg, Wu, sWu, gWu, total_rows, F, K, bias_g,
                           bias_u, act, H, out_dtype, G=None, U=None, stream=None):
    _check(lib().fp4_gemm_gated_grouped(fmt, num_groups, _p(offsets), _p(A), _p(sA), _p(gA), _p(Wg), _p(sWg), _p(gWg),
                                        _p(Wu), _p(sWu), _p(gWu), total_rows, F, K, _p(bias_g), _p(bias_u), act, _p(H),
                                        out_dtype, _p(G), _p(U), _s(stream)))


def fp4_act_backward_workspace_size(rows: int, cols: int, gated: bool) -> int:
    return int(lib().fp4_act_backward_workspace_size(rows, cols, 1 if gated else 0))


def fp4_act_backward(dH, G, U, rows, cols, in_dtype, act, dZ, out_dtype, dbias=None, fmt=NVFP4, codes=None,
                     scales=None, global_in=None, amax_out=None, workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_act_backward(_p(dH), _p(G), _p(U), rows, cols, in_dtype, act, _p(dZ), out_dtype, _p(dbias), fmt,
                                  _p(codes), _p(scales), _p(global_in), _p(amax_out), _p(workspace), workspace_bytes,
                                  _s(stream)))


def fp4_layernorm(x, rows, cols, in_dtype, weight, bias, eps, y, out_dtype, mean=None, rstd=None, fmt=NVFP4,
                  codes=None, scales=None, global_in=None, amax_out=None, stream=None):
    _check(lib().fp4_layernorm(_p(x), rows, cols, in_dtype, _p(weight), _p(bias), eps, _p(y), out_dtype, _p(mean),
                               _p(rstd), fmt, _p(codes), _p(scales), _p(global_in), _p(amax_out), _s(stream)))


def fp4_layernorm_backward_workspace_size(rows: int, cols: int) -> int:
    return int(lib().fp4_layernorm_backward_workspace_size(rows, cols))


def fp4_layernorm_backward(dy, x, rows, cols, in_dtype, weight, mean, rstd, dres, dx, out_dtype, dweight=None,
                           dbias=None, workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_layernorm_backward(_p(dy), _p(x), rows, cols, in_dtype, _p(weight), _p(mean), _p(rstd), _p(dres),
                                        _p(dx), out_dtype, _p(dweight), _p(dbias), _p(workspace), workspace_bytes,
                                        _s(stream)))


def fp4_gemm_noalloc(fmt, A, sA, gA, B, sB, gB, M, N, K, D, out_dtype, stream=None):
    """fp4_gemm without a caller workspace: the split-K scratch is a fixed 4 MiB array
    inside the library, shared by all calls on a device (calls that overlap race)."""
    _check(lib().fp4_gemm_noalloc(fmt, _p(A), _p(sA), _p(gA), _p(B), _p(sB), _p(gB), M, N, K, _p(D), out_dtype,
                                  _s(stream)))


def fp4_gemm_mixed(a_fmt, A, sA, b_fmt, B, sB, M, N, K, D, out_dtype, stream=None):
    """D = A B^T with A and B each MXFP4 or MXFP8 (the FP4 x FP8 GEMM)."""
    _check(lib().fp4_gemm_mixed(a_fmt, _p(A), _p(sA), b_fmt, _p(B), _p(sB), M, N, K, _p(D), out_dtype, _s(stream)))


def fp4_gemm_grouped(fmt, num_groups, offsets, A, sA, gA, B, sB, gB, total_rows, N, K, D, out_dtype,
                     workspace=None, workspace_bytes=0, stream=None):
    _check(lib().fp4_gemm_grouped(fmt, num_groups, _p(offsets), _p(A), _p(sA), _p(gA), _p(B), _p(sB), _p(gB),
                                  total_rows, N, K, _p(D), out_dtype, _p(workspace), workspace_bytes,
                                  _s(stream)))


def fp4_moe_sort_workspace_size(tokens: int, topk: int, num_experts: int) -> int:
    return int(lib().fp4_moe_sort_workspace_size(tokens, topk, num_experts))


def fp4_moe_sort(ids, id_bytes, tokens, topk, num_experts, offsets, row_of, scale_row_of=None, workspace=None,
                 workspace_bytes=0, stream=None):
    _check(lib().fp4_moe_sort(_p(ids), id_bytes, tokens, topk, num_experts, _p(offsets), _p(row_of), _p(scale_row_of),
                              _p(workspace), workspace_bytes, _s(stream)))


def fp4_moe_dispatch(x, tokens, cols, in_dtype, topk, row_of, y, out_dtype, stream=None):
    _check(lib().fp4_moe_dispatch(_p(x), tokens, cols, in_dtype, topk, _p(row_of), _p(y), out_dtype, _s(stream)))


def fp4_moe_dispatch_codes(x, tokens, cols, in_dtype, topk, row_of, scale_row_of, num_experts, offsets, fmt, codes, scales,
                           global_in=None, stream=None):
    _check(lib().fp4_moe_dispatch_codes(_p(x), tokens, cols, in_dtype, topk, _p(row_of), _p(scale_row_of), num_experts,
                                        _p(offsets), fmt, _p(codes), _p(scales), _p(global_in), _s(stream)))


def fp4_moe_dispatch_i8(x, tokens, cols, in_dtype, topk, row_of, codes, row_scales, stream=None):
    _check(lib().fp4_moe_dispatch_i8(_p(x), tokens, cols, in_dtype, topk, _p(row_of), _p(codes), _p(row_scales),
                                     _s(stream)))


def fp4_moe_combine(y, in_dtype, row_of, weights, tokens, topk, cols, residual, residual_dtype, out, out_dtype,
                    stream=None):
    _check(lib().fp4_moe_combine(_p(y), in_dtype, _p(row_of), _p(weights), tokens, topk, cols, _p(residual),
                                 residual_dtype, _p(out), out_dtype, _s(stream)))


def fp4_moe_combine_backward(dout, y, in_dtype, row_of, weights, tokens, topk, cols, dy, out_dtype, dweights=None,
                             stream=None):
    _check(lib().fp4_moe_combine_backward(_p(dout), _p(y), in_dtype, _p(row_of), _p(weights), tokens, topk, cols, _p(dy),
                                          out_dtype, _p(dweights), _s(stream)))


def fp4_quantize_i8(x, rows, cols, in_dtype, codes, row_scales, rows_valid=None, stream=None):
    _check(lib().fp4_quantize_i8(_p(x), rows, cols, in_dtype, _p(codes), _p(row_scales), _p(rows_valid), _s(stream)))


def fp4_gemm_i8_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().fp4_gemm_i8_workspace_size(M, N, K))


def fp4_gemm_i8(A, sA, B, sB, M, N, K, bias, act, D, out_dtype, workspace=None, workspace_bytes=0, flags=0, stream=None):
    _check(lib().fp4_gemm_i8(_p(A), _p(sA), _p(B), _p(sB), M, N, K, _p(bias), act, _p(D), out_dtype, _p(workspace),
                             workspace_bytes, flags, _s(stream)))


def fp4_gemm_i8_grouped_workspace_size(num_groups: int, total_rows: int, N: int, K: int) -> int:
    return int(lib().fp4_gemm_i8_grouped_workspace_size(num_groups, total_rows, N, K))


def fp4_gemm_i8_grouped(num_groups, offsets, A, sA, B, sB, total_rows, N, K, bias, act, D, out_dtype, workspace=None,
                        workspace_bytes=0, stream=None):
    _check(lib().fp4_gemm_i8_grouped(num_groups, _p(offsets), _p(A), _p(sA), _p(B), _p(sB), total_rows, N, K, _p(bias),
                                     act, _p(D), out_dtype, _p(workspace), workspace_bytes, _s(stream)))


def fp4_get_status(stream=None) -> int:
    """Synchronizes the stream and returns (and clears) the latched device status."""
    return int(lib().fp4_get_status(_s(stream)))


def fp4_mma_peak(iters: int, grid: int, cycles, stream=None):
    _check(lib().fp4_mma_peak(iters, grid, _p(cycles), _s(stream)))


def fp4_debug_stall_next_decode(cta: int):
    _check(lib().fp4_debug_stall_next_decode(cta))


def fp4_debug_encode(inp, n, which, out, stream=None):
    _check(lib().fp4_debug_encode(_p(inp), n, which, _p(out), _s(stream)))


# ---------------------------------------------------------------- conveniences
@dataclass
class Quantized:
    """A quantized [rows, cols] tensor in libfp4's layouts (see include/fp4.h)."""
    codes: torch.Tensor                 # uint8 [rows, cols/2]
    scales: torch.Tensor                # uint8, swizzled atoms
    g: torch.Tensor                     # float32 [1] on the device
    rows: int
    cols: int
    fmt: int
    codesT: Optional[torch.Tensor] = None
    scalesT: Optional[torch.Tensor] = None


def _capturing(device: torch.device) -> bool:
    return device.type == "cuda" and torch.cuda.is_current_stream_capturing()


class Workspace:
    """Zero-filled device scratch owned by the caller, reused across calls.

    A buffer that has become too small is kept: captured graphs may still replay calls
    that use it.  Each new one has at least twice its size, so that together they are
    smaller than the buffer in use.  While a graph is being captured the buffer does not
    grow: a call that needs more gets a buffer of its own, zero-filled by every replay (the
    zero-fill of a shared one would wait for the first replay, while other calls already
    use it).  One call of each kind before the capture avoids that."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = torch.zeros(0, dtype=torch.uint8, device=self.device)
        self._outgrown = []

    def get(self, nbytes: int) -> torch.Tensor:
        if nbytes <= self.buf.numel():
            return self.buf
        if _capturing(self.device):
            return torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        new = torch.zeros(max(nbytes, 2 * self.buf.numel(), 4096), dtype=torch.uint8, device=self.device)
        if self.buf.numel():
            self._outgrown.append(self.buf)
        self.buf = new
        return new


def quantize(x: torch.Tensor, fmt: int = NVFP4, block: Optional[int] = None, global_in=None,
             workspace: Optional[Workspace] = None, stream=None) -> Quantized:
    """Allocate outputs and run fp4_quantize on a contiguous [rows, cols] CUDA tensor."""
    if block is None:
        block = 16 if fmt == NVFP4 else 32
    x = x.contiguous()
    rows, cols = (1, x.numel()) if x.dim() == 1 else tuple(x.shape)
    dev = x.device
    codes = torch.empty(rows, cols if fmt == MXFP8 else cols // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(fp4_scales_bytes(rows, cols, fmt), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    codesT = scalesT = None
    if block == 256:
        codesT = torch.empty(cols, rows // 2, dtype=torch.uint8, device=dev)
        scalesT = torch.empty(fp4_scales_bytes(cols, rows, NVFP4), dtype=torch.uint8, device=dev)
    ws = (workspace or Workspace(dev)).get(fp4_quantize_workspace_size())
    fp4_quantize(x, rows, cols, _dtype_code(x), fmt, block, codes, scales, g, codesT, scalesT, global_in, ws,
                 ws.numel(), stream)
    return Quantized(codes, scales, g, rows, cols, fmt, codesT, scalesT)


def gemm(a: Quantized, b: Quantized, out_dtype=torch.bfloat16, workspace: Optional[Workspace] = None,
         stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[M, N] = A . B^T for quantized A [M, K] and B [N, K]."""
    assert a.fmt == b.fmt and a.cols == b.cols
    M, N, K = a.rows, b.rows, a.cols
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=a.codes.device)
    oc = BF16 if out.dtype == torch.bfloat16 else F32
    nbytes = fp4_gemm_workspace_size(M, N, K, a.fmt)
    ws = (workspace or Workspace(a.codes.device)).get(nbytes) if nbytes else None
    fp4_gemm(a.fmt, a.codes, a.scales, a.g, b.codes, b.scales, b.g, M, N, K, out, oc, ws,
             ws.numel() if ws is not None else 0, stream)
    return out


def gemm_mixed(a: Quantized, b: Quantized, out_dtype=torch.bfloat16, stream=None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[M, N] = A . B^T for A and B each quantized as MXFP4 or MXFP8 (K % 128 == 0)."""
    assert a.cols == b.cols
    M, N, K = a.rows, b.rows, a.cols
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=a.codes.device)
    oc = BF16 if out.dtype == torch.bfloat16 else F32
    fp4_gemm_mixed(a.fmt, a.codes, a.scales, b.fmt, b.codes, b.scales, M, N, K, out, oc, stream)
    return out


# ---------------------------------------------------------------- the feed-forward block
# These run on the inputs' device, on `stream` (default: that device's current stream), with
# their outputs allocated on that stream.  Inputs must be dense; biases and norm parameters FP32.
@contextlib.contextmanager
def _on(t: torch.Tensor, stream):
    if not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    with torch.cuda.device(t.device):
        if stream is None:
            yield _s(None)
        elif isinstance(stream, int):
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=t.device)):
                yield stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _dense(name, t, like, shape, dtype=None):
    """Checks an optional operand: on like's device, contiguous, of this shape (and type)."""
    if t is None:
        return
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float32:
        return F32
    raise TypeError(f"output type must be float32 or bfloat16, got {dtype}")


def layernorm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5, out_dtype=None, fmt: Optional[int] = None,
              global_in=None, stream=None, out: Optional[torch.Tensor] = None):
    """Layer norm of the rows of x [rows, cols]: (y, mean, rstd).  With `fmt` (NVFP4, which needs
    the caller's `global_in`, or MXFP4) y is a Quantized tensor instead, without a copy in
    between.  `out` may be x itself."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    rows, cols = x.shape
    _dense("x", x, x, (rows, cols))
    _dense("weight", weight, x, (cols,), torch.float32)
    _dense("bias", bias, x, (cols,), torch.float32)
    _dense("global_in", global_in, x, (1,), torch.float32)
    with _on(x, stream) as s:
        mean, rstd = (torch.empty(rows, dtype=torch.float32, device=x.device) for _ in range(2))
        if fmt is None:
            if out is None:
                out = torch.empty(rows, cols, dtype=out_dtype or x.dtype, device=x.device)
            _dense("out", out, x, (rows, cols))
            fp4_layernorm(x, rows, cols, _dtype_code(x), weight, bias, eps, out, _out_code(out.dtype), mean, rstd, stream=s)
            return out, mean, rstd
        if out is not None or out_dtype is not None:
            raise ValueError("a quantized result takes neither out nor out_dtype")
        codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(fp4_scales_bytes(rows, cols, fmt), dtype=torch.uint8, device=x.device)
        fp4_layernorm(x, rows, cols, _dtype_code(x), weight, bias, eps, None, F32, mean, rstd, fmt, codes, scales,
                      global_in, stream=s)
        g = global_in if fmt == NVFP4 else torch.ones(1, dtype=torch.float32, device=x.device)
        return Quantized(codes, scales, g, rows, cols, fmt), mean, rstd


def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight, mean, rstd, dres=None, out_dtype=None, stream=None):
    """(dx, dweight, dbias) of layernorm; `dres` (x's type) is added to dx."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    rows, cols = x.shape
    _dense("x", x, x, (rows, cols))
    _dense("dy", dy, x, (rows, cols), x.dtype)
    _dense("dres", dres, x, (rows, cols), x.dtype)
    _dense("weight", weight, x, (cols,), torch.float32)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _dense(name, t, x, (rows,), torch.float32)
    with _on(x, stream) as s:
        dx = torch.empty(rows, cols, dtype=out_dtype or x.dtype, device=x.device)
        dw, db = (torch.empty(cols, dtype=torch.float32, device=x.device) for _ in range(2))
        ws = torch.empty(fp4_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=x.device)
        fp4_layernorm_backward(dy, x, rows, cols, _dtype_code(x), weight, mean, rstd, dres, dx, _out_code(dx.dtype), dw,
                               db, ws, ws.numel(), s)
    return dx, dw, db


def gemm_gated(a: Quantized, wg: Quantized, wu: Quantized, act: int = ACT_SILU, bias_g=None, bias_u=None,
               out_dtype=torch.bfloat16, save: bool = False, quantized_out: Optional[torch.Tensor] = None,
               workspace: Optional[Workspace] = None, stream=None):
    """H = act(A . Wg^T + bias_g) * (A . Wu^T + bias_u) [M, F] in one launch; (H, G, U) with
    `save`, which the backward pass needs.  `quantized_out`: the FP32 global scale [1] of an
    NVFP4 result, returned as a Quantized tensor in H's place."""
    if not (a.fmt == wg.fmt == wu.fmt) or not (a.cols == wg.cols == wu.cols) or wg.rows != wu.rows:
        raise ValueError("a, wg and wu must agree in format and columns, wg and wu in rows")
    M, F, K, like = a.rows, wg.rows, a.cols, a.codes
    for name, q in (("wg", wg), ("wu", wu)):
        _dense(f"{name}.codes", q.codes, like, (F, K // 2))
    _dense("bias_g", bias_g, like, (F,), torch.float32)
    _dense("bias_u", bias_u, like, (F,), torch.float32)
    _dense("quantized_out", quantized_out, like, (1,), torch.float32)
    with _on(like, stream) as s:
        def new(dtype=out_dtype):
            return torch.empty(M, F, dtype=dtype, device=like.device)

        H = codes = scales = None
        if quantized_out is None:
            H = new()
        else:
            codes = torch.empty(M, F // 2, dtype=torch.uint8, device=like.device)
            scales = torch.empty(fp4_scales_bytes(M, F, NVFP4), dtype=torch.uint8, device=like.device)
        G, U = (new(), new()) if save else (None, None)
        nbytes = fp4_gemm_gated_workspace_size(M, F, K, a.fmt, codes is not None)
        ws = (workspace or Workspace(like.device)).get(nbytes) if nbytes else None
        fp4_gemm_gated(a.fmt, a.codes, a.scales, a.g, wg.codes, wg.scales, wg.g, wu.codes, wu.scales, wu.g, M, F, K,
                       bias_g, bias_u, act, H, _out_code(out_dtype), G, U, codes, scales, quantized_out, None, ws,
                       ws.numel() if ws is not None else 0, 0, s)
        if codes is not None:
            H = Quantized(codes, scales, quantized_out, M, F, NVFP4)
    return (H, G, U) if save else H


def gemm_epilogue(a: Quantized, b: Quantized, bias=None, act: int = ACT_NONE, residual=None, out_dtype=torch.bfloat16,
                  save: bool = False, workspace: Optional[Workspace] = None, stream=None,
                  out: Optional[torch.Tensor] = None):
    """D = act(A . B^T + bias) + residual; (D, pre-activation) with `save`.  `out` may be the
    residual itself."""
    if a.fmt != b.fmt or a.cols != b.cols:
        raise ValueError("a and b must agree in format and columns")
    M, N, K, like = a.rows, b.rows, a.cols, a.codes
    _dense("b.codes", b.codes, like, (N, K // 2))
    _dense("bias", bias, like, (N,), torch.float32)
    _dense("residual", residual, like, (M, N))
    _dense("out", out, like, (M, N))
    rc = F32 if residual is None else _out_code(residual.dtype)
    with _on(like, stream) as s:
        if out is None:
            out = torch.empty(M, N, dtype=out_dtype, device=like.device)
        pre = torch.empty_like(out) if save else None
        nbytes = fp4_gemm_epilogue_workspace_size(M, N, K, a.fmt, False)
        ws = (workspace or Workspace(like.device)).get(nbytes) if nbytes else None
        fp4_gemm_epilogue_ex(a.fmt, a.codes, a.scales, a.g, b.codes, b.scales, b.g, M, N, K, bias, act, residual, rc, out,
                             _out_code(out.dtype), pre, workspace=ws, workspace_bytes=ws.numel() if ws is not None else 0,
                             stream=s)
    return (out, pre) if save else out


def act_backward(dH: torch.Tensor, G: torch.Tensor, U: Optional[torch.Tensor] = None, act: int = ACT_SILU,
                 dbias: bool = False, out_dtype=None, stream=None):
    """dZ of H = act(G) (U) from dH: [rows, cols], or with U [rows, 2 cols] = [dG | dU]; (dZ,
    its column sums) with `dbias`."""
    if dH.dim() != 2:
        raise ValueError("dH must be [rows, cols]")
    rows, cols = dH.shape
    _dense("dH", dH, dH, (rows, cols))
    _dense("G", G, dH, (rows, cols), dH.dtype)
    _dense("U", U, dH, (rows, cols), dH.dtype)
    width = cols if U is None else 2 * cols
    with _on(dH, stream) as s:
        dZ = torch.empty(rows, width, dtype=out_dtype or dH.dtype, device=dH.device)
        db = ws = None
        if dbias:
            db = torch.empty(width, dtype=torch.float32, device=dH.device)
            ws = torch.empty(fp4_act_backward_workspace_size(rows, cols, U is not None), dtype=torch.uint8, device=dH.device)
        fp4_act_backward(dH, G, U, rows, cols, _dtype_code(dH), act, dZ, _out_code(dZ.dtype), db, workspace=ws,
                         workspace_bytes=ws.numel() if ws is not None else 0, stream=s)
    return (dZ, db) if dbias else dZ


def transposed(w: Quantized) -> Quantized:
    """The W^T operand a 16x16 (block 256) quantization produced alongside W."""
    assert w.codesT is not None
    return Quantized(w.codesT, w.scalesT, w.g, w.cols, w.rows, w.fmt)


# ---------------------------------------------------------------- experts, 8-bit integers
# Devices, streams and density as for the feed-forward block above.
@dataclass
class Routing:
    """Where a router's choices stand in the experts' order (moe_sort)."""
    offsets: torch.Tensor               # int32 [num_experts + 1]
    row_of: torch.Tensor                # int32 [tokens, topk]: a choice's row, -1 for none
    scale_row_of: torch.Tensor          # int32 [tokens, topk]: its row in the grouped scale layout
    num_experts: int

    @property
    def tokens(self) -> int:
        return self.row_of.shape[0]

    @property
    def topk(self) -> int:
        return self.row_of.shape[1]


@dataclass
class Int8Rows:
    """Rows of signed 8-bit integers with one scale each (quantize_i8)."""
    codes: torch.Tensor                 # int8 [rows, cols], weights of experts [experts, rows, cols]
    scales: torch.Tensor                # float32 [rows] or [experts, rows]


def moe_sort(ids: torch.Tensor, num_experts: int, stream=None) -> Routing:
    """Rows of the choices ids [tokens, topk] (int32 or int64) in the experts' order; a number
    outside [0, num_experts) is no expert."""
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, topk]")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    tokens, topk = ids.shape
    _dense("ids", ids, ids, (tokens, topk))
    with _on(ids, stream) as s:
        offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=ids.device)
        row_of, scale_row_of = (torch.empty(tokens, topk, dtype=torch.int32, device=ids.device) for _ in range(2))
        nbytes = fp4_moe_sort_workspace_size(tokens, topk, num_experts)
        # of its own: it needs no zero-fill and leaves none behind
        ws = torch.empty(nbytes, dtype=torch.uint8, device=ids.device) if nbytes else None
        fp4_moe_sort(ids, ids.element_size(), tokens, topk, num_experts, offsets, row_of, scale_row_of, ws, nbytes, s)
    return Routing(offsets, row_of, scale_row_of, num_experts)


def _routed(r: Routing, like: torch.Tensor):
    _dense("offsets", r.offsets, like, (r.num_experts + 1,), torch.int32)
    for name, t in (("row_of", r.row_of), ("scale_row_of", r.scale_row_of)):
        _dense(name, t, like, (r.tokens, r.topk), torch.int32)


def moe_dispatch(x: torch.Tensor, routing: Routing, fmt: Optional[int] = None, global_in=None, out_dtype=None, stream=None):
    """The rows of x [tokens, cols] in the experts' order, [tokens * topk, cols]; rows behind the
    last expert's hold nothing.  With `fmt` (NVFP4, which needs the caller's `global_in`, or MXFP4) a
    Quantized tensor with grouped scales instead, the A operand of the grouped products."""
    tokens, cols = routing.tokens, x.shape[-1]
    _dense("x", x, x, (tokens, cols))
    _routed(routing, x)
    _dense("global_in", global_in, x, (1,), torch.float32)
    rows = tokens * routing.topk
    with _on(x, stream) as s:
        if fmt is None:
            y = torch.empty(rows, cols, dtype=out_dtype or x.dtype, device=x.device)
            fp4_moe_dispatch(x, tokens, cols, _dtype_code(x), routing.topk, routing.row_of, y, _out_code(y.dtype), s)
            return y
        if out_dtype is not None:
            raise ValueError("a quantized result takes no out_dtype")
        codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(fp4_scales_bytes_grouped(rows, routing.num_experts, cols, fmt), dtype=torch.uint8,
                             device=x.device)
        fp4_moe_dispatch_codes(x, tokens, cols, _dtype_code(x), routing.topk, routing.row_of, routing.scale_row_of,
                               routing.num_experts, routing.offsets, fmt, codes, scales, global_in, s)
        g = global_in if fmt == NVFP4 else torch.ones(1, dtype=torch.float32, device=x.device)
        return Quantized(codes, scales, g, rows, cols, fmt)


def moe_dispatch_i8(x: torch.Tensor, routing: Routing, stream=None) -> Int8Rows:
    """The rows of x [tokens, cols] in the experts' order as 8-bit rows (cols % 16 == 0)."""
    tokens, cols = routing.tokens, x.shape[-1]
    _dense("x", x, x, (tokens, cols))
    _routed(routing, x)
    with _on(x, stream) as s:
        codes = torch.empty(tokens * routing.topk, cols, dtype=torch.int8, device=x.device)
        scales = torch.empty(tokens * routing.topk, dtype=torch.float32, device=x.device)
        fp4_moe_dispatch_i8(x, tokens, cols, _dtype_code(x), routing.topk, routing.row_of, codes, scales, s)
    return Int8Rows(codes, scales)


def moe_combine(y: torch.Tensor, routing: Routing, weights=None, residual=None, out_dtype=None, stream=None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum over t's choices of weight * y[its row] + residual[t]; weights [tokens, topk]
    FP32, or 1 each.  `out` may be the residual itself."""
    tokens, cols = routing.tokens, y.shape[-1]
    _dense("y", y, y, (tokens * routing.topk, cols))
    _routed(routing, y)
    _dense("weights", weights, y, (tokens, routing.topk), torch.float32)
    _dense("residual", residual, y, (tokens, cols))
    _dense("out", out, y, (tokens, cols))
    rc = F32 if residual is None else _out_code(residual.dtype)
    with _on(y, stream) as s:
        if out is None:
            out = torch.empty(tokens, cols, dtype=out_dtype or y.dtype, device=y.device)
        fp4_moe_combine(y, _dtype_code(y), routing.row_of, weights, tokens, routing.topk, cols, residual, rc, out,
                        _out_code(out.dtype), s)
    return out


def moe_dispatch_backward(dy: torch.Tensor, routing: Routing, out_dtype=None, stream=None) -> torch.Tensor:
    """dx of moe_dispatch: the sum of dy over a token's rows."""
    return moe_combine(dy, routing, out_dtype=out_dtype, stream=stream)


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, routing: Routing, weights=None, out_dtype=None, stream=None):
    """(dy, dweights) of moe_combine (rows of dy behind the last expert's hold nothing); the
    residual's gradient is dout itself."""
    tokens, cols = routing.tokens, y.shape[-1]
    _dense("y", y, y, (tokens * routing.topk, cols))
    _dense("dout", dout, y, (tokens, cols), y.dtype)
    _routed(routing, y)
    _dense("weights", weights, y, (tokens, routing.topk), torch.float32)
    with _on(y, stream) as s:
        dy = torch.empty(tokens * routing.topk, cols, dtype=out_dtype or y.dtype, device=y.device)
        dw = torch.empty(tokens, routing.topk, dtype=torch.float32, device=y.device)
        fp4_moe_combine_backward(dout, y, _dtype_code(y), routing.row_of, weights, tokens, routing.topk, cols, dy,
                                 _out_code(dy.dtype), dw, s)
    return dy, dw


def quantize_i8(x: torch.Tensor, offsets: Optional[torch.Tensor] = None, stream=None) -> Int8Rows:
    """Rows of x [rows, cols] (cols % 16 == 0), or of experts' weights [experts, rows, cols], as
    8-bit integers with one scale each.  With `offsets` (Routing.offsets) x holds rows in the
    experts' order, and those behind the last expert's are left out."""
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, cols] or [experts, rows, cols]")
    _dense("x", x, x, x.shape)
    if offsets is not None:
        _dense("offsets", offsets, x, (offsets.numel(),), torch.int32)
        if offsets.numel() < 2:  # (an empty tensor's address is none, which would mean all rows)
            raise ValueError("offsets must be [experts + 1]")
    rows, cols = x.numel() // max(1, x.shape[-1]), x.shape[-1]
    with _on(x, stream) as s:
        codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        fp4_quantize_i8(x, rows, cols, _dtype_code(x), codes, scales, None if offsets is None else offsets[-1:], s)
    return Int8Rows(codes, scales)


def gemm_i8(a: Int8Rows, b: Int8Rows, bias=None, act: int = ACT_NONE, out_dtype=torch.bfloat16, offsets=None,
            workspace: Optional[Workspace] = None, stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """D[M, N] = act(A . B^T + bias) in 8-bit integers.  With `offsets` (Routing.offsets) rows of A
    sorted by expert, each with its expert's weights b [experts, N, K] and bias [experts, N]; rows of
    D behind the last expert's are left as they were (`out`) or hold nothing."""
    experts = () if offsets is None else (b.codes.shape[0],)
    if a.codes.dim() != 2 or b.codes.dim() != 2 + len(experts) or a.codes.shape[1] != b.codes.shape[-1]:
        raise ValueError("a must be [M, K] and b [N, K], with offsets [experts, N, K]")
    (M, K), N, like = a.codes.shape, b.codes.shape[-2], a.codes
    _dense("a.codes", a.codes, like, (M, K), torch.int8)
    _dense("a.scales", a.scales, like, (M,), torch.float32)
    _dense("b.codes", b.codes, like, (*experts, N, K), torch.int8)
    _dense("b.scales", b.scales, like, (*experts, N), torch.float32)
    _dense("bias", bias, like, (*experts, N), torch.float32)
    _dense("out", out, like, (M, N))
    if experts:
        _dense("offsets", offsets, like, (experts[0] + 1,), torch.int32)
    with _on(like, stream) as s:
        if out is None:
            out = torch.empty(M, N, dtype=out_dtype, device=like.device)
        nbytes = (fp4_gemm_i8_grouped_workspace_size(experts[0], M, N, K) if experts
                  else fp4_gemm_i8_workspace_size(M, N, K))
        ws = (workspace or Workspace(like.device)).get(nbytes) if nbytes else None
        size = ws.numel() if ws is not None else 0
        if experts:
            fp4_gemm_i8_grouped(experts[0], offsets, a.codes, a.scales, b.codes, b.scales, M, N, K, bias, act, out,
                                _out_code(out.dtype), ws, size, s)
        else:
            fp4_gemm_i8(a.codes, a.scales, b.codes, b.scales, M, N, K, bias, act, out, _out_code(out.dtype), ws, size, 0, s)
    return out
