"""ctypes binding of libmx355.so (include/mx.h) and of the workload generator
libmx355_synth.so (include/mx_synth.h).

Argument marshalling only: every step of the hot path runs in the HIP library.
The functions named like the C entry points take torch tensors (device memory)
and the current torch stream; they raise MxError on a non-zero status.  The
library is loaded on first use and a missing build raises immediately -- there
is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from pathlib import Path

import torch

MX_OK, MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_ENUM, MX_ERR_WORKSPACE, MX_ERR_HIP = range(7)
MX_F32, MX_BF16 = 0, 1
MX_ROW, MX_COL = 0, 1
MX_RNE, MX_SR = 0, 1
MX_I32, MX_I64 = 0, 1
MX_SILU, MX_GELU = 0, 1
MX_MAX_GROUPS = 128

LIB_PATH = Path(__file__).resolve().parent / "libmx355.so"
SYNTH_LIB_PATH = Path(__file__).resolve().parent / "libmx355_synth.so"

_c_void_p, _i64, _u64, _u32, _i32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64,
                                                  ctypes.c_uint32, ctypes.c_int, ctypes.c_float,
                                                  ctypes.c_size_t)
_P = _c_void_p
SIGNATURES = {
    "mx_status_string": ([_i32], ctypes.c_char_p),
    "mx_quantize": ([_P, _i32, _i64, _i64, _i32, _i32, _u64, _i32, _u32, _P, _P, _P], _i32),
    "mx_quantize_ld": ([_P, _i32, _i64, _i64, _i32, _i32, _u64, _i32, _u32, _P, _P, _i64, _P], _i32),
    "mx_quantize_dual": ([_P, _i32, _i64, _i64, _i32, _u64, _u64, _P, _P, _P, _P, _P], _i32),
    "mx_requantize": ([_P, _P, _i64, _i64, _i32, _u64, _P, _P, _P], _i32),
    "mx_quantize_pair": ([_P, _i64, _P, _i64, _i64, _i32, _i32, _u64, _u64, _i32, _u32,
                          _P, _P, _P, _P, _P], _i32),
    "mx_requantize_pair": ([_P, _P, _i64, _P, _P, _i64, _i64, _i32, _u64, _u64,
                            _P, _P, _P, _P, _P], _i32),
    "mx_quantize_dual_rht": ([_P, _i32, _i64, _i64, _i32, _u64, _u64, _u32, _P, _P, _P, _P, _P], _i32),
    "mx_requantize_rht": ([_P, _P, _i64, _i64, _i32, _u64, _u32, _P, _P, _P], _i32),
    "mx_segments_padded_rows": ([_P, _i64], _i64),
    "mx_quantize_segments": ([_P, _i32, _i64, _i64, _P, _i64, _i32, _u64, _P, _P, _P], _i32),
    "mx_requantize_segments": ([_P, _P, _i64, _i64, _P, _i64, _i32, _u64, _P, _P, _P], _i32),
    "mx_dequantize": ([_P, _P, _i64, _i64, _i32, _i32, _u32, _P, _i32, _P], _i32),
    "mx_gemm": ([_P, _P, _P, _P, _i64, _i64, _i64, _f32, _P, _i64, _P], _i32),
    "mx_gemm_grouped": ([_P, _P, _P, _P, _P, _i64, _i64, _i64, _f32, _P, _P], _i32),
    "mx_gemm_ld": ([_P, _P, _i64, _P, _P, _i64, _i64, _i64, _i64, _f32, _P, _i64, _P], _i32),
    "mx_gemm_grouped_ld": ([_P, _P, _i64, _P, _P, _i64, _P, _i64, _i64, _i64, _f32, _P, _P], _i32),
    "mx_linear_fwd": ([_P, _P, _i32, _i64, _i64, _i64, _P, _P, _P, _P, _P, _P], _i32),
    "mx_linear_bwd_workspace_size": ([_i64, _i64, _i64], _sz),
    "mx_linear_bwd": ([_P, _i32, _i64, _i64, _i64, _P, _P, _P, _P, _u64, _P, _P, _P, _sz, _P], _i32),
    "mx_linear_bwd_noalloc": ([_P, _i32, _i64, _i64, _i64, _P, _P, _P, _P, _u64, _P, _P, _P], _i32),
    "mx_linear_bwd_noalloc_max_workspace": ([], _sz),
    "mx_grouped_linear_bwd_workspace_size": ([_P, _i64, _i64, _i64], _sz),
    "mx_grouped_linear_bwd": ([_P, _i32, _P, _i64, _i64, _i64, _P, _P, _P, _P, _u64, _P, _P, _P, _sz,
                               _P], _i32),
    "mx_linear_fwd_rht": ([_P, _P, _i32, _i64, _i64, _i64, _u32, _P, _P, _P, _P, _P, _P], _i32),
    "mx_linear_bwd_rht": ([_P, _i32, _i64, _i64, _i64, _P, _P, _P, _P, _u64, _u32, _P, _P, _P, _sz,
                           _P], _i32),
    "mx_gemv_workspace_size": ([_i32, _i64, _i64, _i64], _sz),
    "mx_gemv": ([_P, _i32, _i64, _P, _P, _i64, _i64, _i64, _i64, _f32, _P, _i32, _i64, _P, _sz, _P],
                _i32),
    "mx_gemv_grouped": ([_P, _i32, _i64, _i64, _P, _i64, _P, _P, _i64, _P, _i64, _i64, _i64, _i64,
                         _f32, _P, _i32, _i64, _P], _i32),
    "mx_moe_plan_workspace_size": ([_i64, _i64, _i64], _sz),
    "mx_moe_plan": ([_P, _i32, _i64, _i64, _i64, _P, _P, _P, _P, _sz, _P], _i32),
    "mx_moe_dispatch": ([_P, _i32, _i64, _P, _P, _i64, _i64, _i64, _i64, _P, _i64, _P], _i32),
    "mx_moe_dispatch_quantize": ([_P, _i32, _i64, _P, _i64, _i64, _i64, _i64, _P, _P, _i64, _P], _i32),
    "mx_moe_combine": ([_P, _i32, _i64, _i64, _P, _P, _i64, _i64, _i64, _P, _i32, _i64, _P], _i32),
    "mx_moe_combine_bwd": ([_P, _i32, _i64, _P, _i32, _i64, _i64, _P, _P, _i64, _i64, _i64, _P, _i64,
                            _P, _P], _i32),
    "mx_quantize8": ([_P, _i32, _i64, _i64, _i64, _i32, _P, _i64, _P, _i64, _P], _i32),
    "mx_quantize8_dual": ([_P, _i32, _i64, _i64, _i64, _i32, _P, _i64, _P, _i64, _P, _i64, _P, _i64, _P], _i32),
    "mx_requantize8": ([_P, _i64, _P, _i64, _i64, _i64, _P, _i64, _P, _i64, _P], _i32),
    "mx_dequantize8": ([_P, _i64, _P, _i64, _i64, _i64, _P, _i32, _i64, _P], _i32),
    "mx_gemm8_workspace_size": ([_i64, _i64, _i64], _sz),
    "mx_gemm8": ([_P, _i64, _P, _i64, _P, _i64, _P, _i64, _i64, _i64, _i64, _f32, _P, _i32, _i64, _P, _sz, _P],
                 _i32),
    "mx_linear8_fwd_workspace_size": ([_i64, _i64, _i64], _sz),
    "mx_linear8_fwd": ([_P, _i32, _i64, _P, _i32, _i64, _i64, _i64, _i64, _P, _i32, _i64, _P, _P, _P, _P, _P, _P,
                        _P, _sz, _P], _i32),
    "mx_linear8_bwd_workspace_size": ([_i64, _i64, _i64], _sz),
    "mx_linear8_bwd": ([_P, _i32, _i64, _i64, _i64, _i64, _P, _P, _P, _P, _P, _i32, _i64, _P, _i64, _P, _sz, _P],
                       _i32),
    "mx_glu": ([_P, _i32, _i64, _P, _i64, _i64, _i32, _P, _i32, _i64, _P, _i64, _P, _i64, _P], _i32),
    "mx_glu_quantize": ([_P, _i32, _i64, _P, _i64, _i64, _i32, _P, _P, _i64, _P, _i64, _P, _i64, _P], _i32),
    "mx_glu_quantize8": ([_P, _i32, _i64, _P, _i64, _i64, _i32, _P, _i64, _P, _i64, _P, _i64, _P, _i64, _P], _i32),
    "mx_glu_bwd": ([_P, _i32, _i64, _P, _i64, _P, _i64, _P, _i64, _i64, _i32, _P, _i32, _i64, _P], _i32),
    "mx_moe_route_workspace_size": ([_i64, _i64, _i64], _sz),
    "mx_moe_route": ([_P, _i32, _i64, _P, _i64, _i64, _i64, _i32, _P, _P, _P, _P, _P, _P, _sz, _P], _i32),
    "mx_moe_route_bwd": ([_P, _i32, _i64, _P, _i64, _i64, _i64, _i32, _P, _P, _P, _P, _P, _i64, _P], _i32),
    "mx_deosc_init": ([_P, _i64, _i64, _P, _P, _P, _P], _i32),
    "mx_deosc_step": ([_P, _i64, _i64, _P, _P, _P, _i32, _f32, _P, _P], _i32),
    "mx_deosc_step_quantize": ([_P, _i64, _i64, _P, _P, _P, _i32, _f32, _P, _P, _P, _P], _i32),
    "mx_qema_step": ([_P, _P, _i64, _i64, _f32, _P, _P, _P], _i32),
}
SYNTH_SIGNATURES = {
    "mx_synth_step": ([_P, _i64, _u64, _i64, _P], _i32),
}

_lib = None
_synth_lib = None


class MxError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} -> {status_string(status)}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mxfp4_microscaling_quantization_amd.build`")
        handle = ctypes.CDLL(str(LIB_PATH))
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def synth_lib() -> ctypes.CDLL:
    """The workload generator's library (the synthetic optimizer steps); raises if
    it has not been built."""
    global _synth_lib
    if _synth_lib is None:
        if not SYNTH_LIB_PATH.exists():
            raise RuntimeError(f"{SYNTH_LIB_PATH} is missing: build it with "
                               "`python -m mxfp4_microscaling_quantization_amd.build`")
        handle = ctypes.CDLL(str(SYNTH_LIB_PATH))
        for name, (args, res) in SYNTH_SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _synth_lib = handle
    return _synth_lib


def status_string(status: int) -> str:
    return lib().mx_status_string(int(status)).decode()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # the handle alone: a Stream object costs 2.6 us more
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name: str, status: int) -> None:
    if status != MX_OK:
        raise MxError(name, status)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MX_F32
    if t.dtype == torch.bfloat16:
        return MX_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------ C-named entry points
def mx_quantize(x, dtype, rows, cols, axis, round, seed, hadamard, sign_mask, codes, scales,
                stream=None):
    _check("mx_quantize", lib().mx_quantize(_ptr(x), dtype, rows, cols, axis, round, seed,
                                            hadamard, sign_mask, _ptr(codes), _ptr(scales),
                                            _stream(stream)))


def mx_quantize_ld(x, dtype, rows, cols, axis, round, seed, hadamard, sign_mask, codes, scales,
                   scale_ld, stream=None):
    _check("mx_quantize_ld", lib().mx_quantize_ld(_ptr(x), dtype, rows, cols, axis, round, seed,
                                                  hadamard, sign_mask, _ptr(codes), _ptr(scales),
                                                  scale_ld, _stream(stream)))


def mx_quantize_dual(x, dtype, rows, cols, round, seed_row, seed_col, codes_row, scales_row,
                     codes_col, scales_col, stream=None):
    _check("mx_quantize_dual", lib().mx_quantize_dual(
        _ptr(x), dtype, rows, cols, round, seed_row, seed_col, _ptr(codes_row), _ptr(scales_row),
        _ptr(codes_col), _ptr(scales_col), _stream(stream)))


def mx_quantize_dual_rht(x, dtype, rows, cols, round, seed_row, seed_col, sign_mask, codes_row,
                         scales_row, codes_col, scales_col, stream=None):
    _check("mx_quantize_dual_rht", lib().mx_quantize_dual_rht(
        _ptr(x), dtype, rows, cols, round, seed_row, seed_col, sign_mask, _ptr(codes_row),
        _ptr(scales_row), _ptr(codes_col), _ptr(scales_col), _stream(stream)))


def mx_requantize_rht(codes_in, scales_in, rows, cols, round, seed, sign_mask, codes_out,
                      scales_out, stream=None):
    _check("mx_requantize_rht", lib().mx_requantize_rht(
        _ptr(codes_in), _ptr(scales_in), rows, cols, round, seed, sign_mask, _ptr(codes_out),
        _ptr(scales_out), _stream(stream)))


def mx_requantize(codes_in, scales_in, rows, cols, round, seed, codes_out, scales_out, stream=None):
    _check("mx_requantize", lib().mx_requantize(_ptr(codes_in), _ptr(scales_in), rows, cols, round,
                                                seed, _ptr(codes_out), _ptr(scales_out),
                                                _stream(stream)))


def mx_quantize_pair(x0, rows0, x1, rows1, cols, dtype, round, seed0, seed1, hadamard, sign_mask,
                     codes0, scales0, codes1, scales1, stream=None):
    _check("mx_quantize_pair", lib().mx_quantize_pair(
        _ptr(x0), rows0, _ptr(x1), rows1, cols, dtype, round, seed0, seed1, hadamard, sign_mask,
        _ptr(codes0), _ptr(scales0), _ptr(codes1), _ptr(scales1), _stream(stream)))


def mx_requantize_pair(codes_in0, scales_in0, rows0, codes_in1, scales_in1, rows1, cols, round,
                       seed0, seed1, codes_out0, scales_out0, codes_out1, scales_out1,
                       stream=None):
    _check("mx_requantize_pair", lib().mx_requantize_pair(
        _ptr(codes_in0), _ptr(scales_in0), rows0, _ptr(codes_in1), _ptr(scales_in1), rows1, cols,
        round, seed0, seed1, _ptr(codes_out0), _ptr(scales_out0), _ptr(codes_out1),
        _ptr(scales_out1), _stream(stream)))


def mx_dequantize(codes, scales, rows, cols, axis, hadamard, sign_mask, out, out_dtype,
                  stream=None):
    _check("mx_dequantize", lib().mx_dequantize(_ptr(codes), _ptr(scales), rows, cols, axis,
                                                hadamard, sign_mask, _ptr(out), out_dtype,
                                                _stream(stream)))


def mx_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, alpha, c, ldc, stream=None):
    _check("mx_gemm", lib().mx_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales),
                                    M, N, K, alpha, _ptr(c), ldc, _stream(stream)))


def mx_gemm_ld(a_codes, a_scales, a_scale_ld, b_codes, b_scales, b_scale_ld, M, N, K, alpha, c,
               ldc, stream=None):
    _check("mx_gemm_ld", lib().mx_gemm_ld(_ptr(a_codes), _ptr(a_scales), a_scale_ld,
                                          _ptr(b_codes), _ptr(b_scales), b_scale_ld, M, N, K,
                                          alpha, _ptr(c), ldc, _stream(stream)))


def _offsets(offs):
    """Host int64 array of the offsets (kept alive by the caller's reference)."""
    return (ctypes.c_int64 * len(offs))(*[int(o) for o in offs])


def mx_segments_padded_rows(offs, groups) -> int:
    arr = _offsets(offs)
    return int(lib().mx_segments_padded_rows(ctypes.addressof(arr), groups))


def mx_quantize_segments(x, dtype, rows, cols, offs, groups, round, seed, codes, scales,
                         stream=None):
    arr = _offsets(offs)
    _check("mx_quantize_segments", lib().mx_quantize_segments(
        _ptr(x), dtype, rows, cols, ctypes.addressof(arr), groups, round, seed, _ptr(codes),
        _ptr(scales), _stream(stream)))


def mx_requantize_segments(codes_in, scales_in, rows, cols, offs, groups, round, seed, codes_out,
                           scales_out, stream=None):
    arr = _offsets(offs)
    _check("mx_requantize_segments", lib().mx_requantize_segments(
        _ptr(codes_in), _ptr(scales_in), rows, cols, ctypes.addressof(arr), groups, round, seed,
        _ptr(codes_out), _ptr(scales_out), _stream(stream)))


def mx_grouped_linear_bwd_workspace_size(offs, groups, N, K) -> int:
    arr = _offsets(offs)
    return int(lib().mx_grouped_linear_bwd_workspace_size(ctypes.addressof(arr), groups, N, K))


def mx_grouped_linear_bwd(dy, dtype, offs, groups, N, K, xq_codes, xq_scales, wq_codes, wq_scales,
                          seed, dx, dw, workspace, workspace_bytes, stream=None):
    arr = _offsets(offs)
    _check("mx_grouped_linear_bwd", lib().mx_grouped_linear_bwd(
        _ptr(dy), dtype, ctypes.addressof(arr), groups, N, K, _ptr(xq_codes), _ptr(xq_scales),
        _ptr(wq_codes), _ptr(wq_scales), seed, _ptr(dx), _ptr(dw), _ptr(workspace),
        workspace_bytes, _stream(stream)))


def mx_gemm_grouped(a_codes, a_scales, b_codes, b_scales, offs, groups, N, K, alpha, c,
                    stream=None):
    arr = _offsets(offs)
    _check("mx_gemm_grouped", lib().mx_gemm_grouped(
        _ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), ctypes.addressof(arr),
        groups, N, K, alpha, _ptr(c), _stream(stream)))


def mx_gemm_grouped_ld(a_codes, a_scales, a_scale_ld, b_codes, b_scales, b_scale_ld, offs, groups,
                       N, K, alpha, c, stream=None):
    arr = _offsets(offs)
    _check("mx_gemm_grouped_ld", lib().mx_gemm_grouped_ld(
        _ptr(a_codes), _ptr(a_scales), a_scale_ld, _ptr(b_codes), _ptr(b_scales), b_scale_ld,
        ctypes.addressof(arr), groups, N, K, alpha, _ptr(c), _stream(stream)))


def mx_linear_fwd(x, w, dtype, M, N, K, y, xq_codes, xq_scales, wq_codes, wq_scales, stream=None):
    _check("mx_linear_fwd", lib().mx_linear_fwd(_ptr(x), _ptr(w), dtype, M, N, K, _ptr(y),
                                                _ptr(xq_codes), _ptr(xq_scales), _ptr(wq_codes),
                                                _ptr(wq_scales), _stream(stream)))


def mx_linear_fwd_rht(x, w, dtype, M, N, K, sign_mask, y, xq_codes, xq_scales, wq_codes,
                      wq_scales, stream=None):
    _check("mx_linear_fwd_rht", lib().mx_linear_fwd_rht(
        _ptr(x), _ptr(w), dtype, M, N, K, sign_mask, _ptr(y), _ptr(xq_codes), _ptr(xq_scales),
        _ptr(wq_codes), _ptr(wq_scales), _stream(stream)))


def mx_linear_bwd_workspace_size(M, N, K) -> int:
    return int(lib().mx_linear_bwd_workspace_size(M, N, K))


def mx_linear_bwd(dy, dtype, M, N, K, xq_codes, xq_scales, wq_codes, wq_scales, seed, dx, dw,
                  workspace, workspace_bytes, stream=None):
    _check("mx_linear_bwd", lib().mx_linear_bwd(
        _ptr(dy), dtype, M, N, K, _ptr(xq_codes), _ptr(xq_scales), _ptr(wq_codes),
        _ptr(wq_scales), seed, _ptr(dx), _ptr(dw), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def mx_linear_bwd_noalloc(dy, dtype, M, N, K, xq_codes, xq_scales, wq_codes, wq_scales, seed, dx,
                          dw, stream=None):
    _check("mx_linear_bwd_noalloc", lib().mx_linear_bwd_noalloc(
        _ptr(dy), dtype, M, N, K, _ptr(xq_codes), _ptr(xq_scales), _ptr(wq_codes),
        _ptr(wq_scales), seed, _ptr(dx), _ptr(dw), _stream(stream)))


def mx_linear_bwd_noalloc_max_workspace():
    return int(lib().mx_linear_bwd_noalloc_max_workspace())


def mx_linear_bwd_rht(dy, dtype, M, N, K, xq_codes, xq_scales, wq_codes, wq_scales, seed,
                      sign_mask, dx, dw, workspace, workspace_bytes, stream=None):
    _check("mx_linear_bwd_rht", lib().mx_linear_bwd_rht(
        _ptr(dy), dtype, M, N, K, _ptr(xq_codes), _ptr(xq_scales), _ptr(wq_codes),
        _ptr(wq_scales), seed, sign_mask, _ptr(dx), _ptr(dw), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def mx_gemv_workspace_size(x_dtype, M, N, K) -> int:
    return int(lib().mx_gemv_workspace_size(x_dtype, M, N, K))


def mx_gemv(x, x_dtype, ldx, w_codes, w_scales, w_scale_ld, M, N, K, alpha, y, y_dtype, ldy,
            workspace=None, workspace_bytes=0, stream=None):
    _check("mx_gemv", lib().mx_gemv(_ptr(x), x_dtype, ldx, _ptr(w_codes), _ptr(w_scales), w_scale_ld,
                                    M, N, K, alpha, _ptr(y), y_dtype, ldy, _ptr(workspace),
                                    workspace_bytes, _stream(stream)))


def mx_gemv_grouped(x, x_dtype, ldx, x_rows, src, top_k, w_codes, w_scales, w_scale_ld, offs, groups,
                    rows, N, K, alpha, y, y_dtype, ldy, stream=None):
    _check("mx_gemv_grouped", lib().mx_gemv_grouped(
        _ptr(x), x_dtype, ldx, x_rows, _ptr(src), top_k, _ptr(w_codes), _ptr(w_scales), w_scale_ld,
        _ptr(offs), groups, rows, N, K, alpha, _ptr(y), y_dtype, ldy, _stream(stream)))


def mx_moe_plan_workspace_size(tokens, top_k, experts) -> int:
    return int(lib().mx_moe_plan_workspace_size(tokens, top_k, experts))


def mx_moe_plan(ids, id_type, tokens, top_k, experts, offs, src, pos, workspace, workspace_bytes,
                stream=None):
    _check("mx_moe_plan", lib().mx_moe_plan(_ptr(ids), id_type, tokens, top_k, experts, _ptr(offs),
                                            _ptr(src), _ptr(pos), _ptr(workspace), workspace_bytes,
                                            _stream(stream)))


def mx_moe_dispatch(x, dtype, ldx, pos, weights, tokens, top_k, rows, cols, out, ldo, stream=None):
    _check("mx_moe_dispatch", lib().mx_moe_dispatch(
        _ptr(x), dtype, ldx, _ptr(pos), _ptr(weights), tokens, top_k, rows, cols, _ptr(out), ldo,
        _stream(stream)))


def mx_moe_dispatch_quantize(x, dtype, ldx, pos, tokens, top_k, rows, cols, codes, scales, scale_ld,
                             stream=None):
    _check("mx_moe_dispatch_quantize", lib().mx_moe_dispatch_quantize(
        _ptr(x), dtype, ldx, _ptr(pos), tokens, top_k, rows, cols, _ptr(codes), _ptr(scales),
        scale_ld, _stream(stream)))


def mx_moe_combine(z, z_dtype, ldz, rows, pos, weights, tokens, top_k, cols, y, y_dtype, ldy,
                   stream=None):
    _check("mx_moe_combine", lib().mx_moe_combine(
        _ptr(z), z_dtype, ldz, rows, _ptr(pos), _ptr(weights), tokens, top_k, cols, _ptr(y), y_dtype,
        ldy, _stream(stream)))


def mx_moe_combine_bwd(dy, dy_dtype, lddy, z, z_dtype, ldz, rows, pos, weights, tokens, top_k, cols,
                       dz, lddz, dweights, stream=None):
    _check("mx_moe_combine_bwd", lib().mx_moe_combine_bwd(
        _ptr(dy), dy_dtype, lddy, _ptr(z), z_dtype, ldz, rows, _ptr(pos), _ptr(weights), tokens,
        top_k, cols, _ptr(dz), lddz, _ptr(dweights), _stream(stream)))


def mx_quantize8(x, dtype, ldx, rows, cols, axis, codes, ld, scales, scale_ld, stream=None):
    _check("mx_quantize8", lib().mx_quantize8(_ptr(x), dtype, ldx, rows, cols, axis, _ptr(codes), ld,
                                              _ptr(scales), scale_ld, _stream(stream)))


def mx_quantize8_dual(x, dtype, ldx, rows, cols, tile, codes, ld, scales, scale_ld, codes_t, ld_t, scales_t,
                      scale_ld_t, stream=None):
    _check("mx_quantize8_dual", lib().mx_quantize8_dual(
        _ptr(x), dtype, ldx, rows, cols, tile, _ptr(codes), ld, _ptr(scales), scale_ld, _ptr(codes_t), ld_t,
        _ptr(scales_t), scale_ld_t, _stream(stream)))


def mx_requantize8(codes, ld, scales, scale_ld, rows, cols, codes_t, ld_t, scales_t, scale_ld_t, stream=None):
    _check("mx_requantize8", lib().mx_requantize8(
        _ptr(codes), ld, _ptr(scales), scale_ld, rows, cols, _ptr(codes_t), ld_t, _ptr(scales_t), scale_ld_t,
        _stream(stream)))


def mx_dequantize8(codes, ld, scales, scale_ld, rows, cols, out, out_dtype, ldo, stream=None):
    _check("mx_dequantize8", lib().mx_dequantize8(_ptr(codes), ld, _ptr(scales), scale_ld, rows, cols, _ptr(out),
                                                  out_dtype, ldo, _stream(stream)))


def mx_gemm8_workspace_size(M, N, K) -> int:
    return int(lib().mx_gemm8_workspace_size(M, N, K))


def mx_gemm8(a_codes, lda, a_scales, a_scale_ld, b_codes, ldb, b_scales, b_scale_ld, M, N, K, alpha, c, c_dtype,
             ldc, workspace=None, workspace_bytes=0, stream=None):
    _check("mx_gemm8", lib().mx_gemm8(
        _ptr(a_codes), lda, _ptr(a_scales), a_scale_ld, _ptr(b_codes), ldb, _ptr(b_scales), b_scale_ld, M, N, K,
        alpha, _ptr(c), c_dtype, ldc, _ptr(workspace), workspace_bytes, _stream(stream)))


def mx_linear8_fwd_workspace_size(M, N, K) -> int:
    return int(lib().mx_linear8_fwd_workspace_size(M, N, K))


def mx_linear8_fwd(x, x_dtype, ldx, w, w_dtype, ldw, M, N, K, y, y_dtype, ldy, xq_codes, xq_scales, wq_codes,
                   wq_scales, wt_codes, wt_scales, workspace=None, workspace_bytes=0, stream=None):
    _check("mx_linear8_fwd", lib().mx_linear8_fwd(
        _ptr(x), x_dtype, ldx, _ptr(w), w_dtype, ldw, M, N, K, _ptr(y), y_dtype, ldy, _ptr(xq_codes),
        _ptr(xq_scales), _ptr(wq_codes), _ptr(wq_scales), _ptr(wt_codes), _ptr(wt_scales), _ptr(workspace),
        workspace_bytes, _stream(stream)))


def mx_linear8_bwd_workspace_size(M, N, K) -> int:
    return int(lib().mx_linear8_bwd_workspace_size(M, N, K))


def mx_linear8_bwd(dy, dy_dtype, lddy, M, N, K, xq_codes, xq_scales, wt_codes, wt_scales, dx, dx_dtype, lddx, dw,
                   lddw, workspace, workspace_bytes, stream=None):
    _check("mx_linear8_bwd", lib().mx_linear8_bwd(
        _ptr(dy), dy_dtype, lddy, M, N, K, _ptr(xq_codes), _ptr(xq_scales), _ptr(wt_codes), _ptr(wt_scales),
        _ptr(dx), dx_dtype, lddx, _ptr(dw), lddw, _ptr(workspace), workspace_bytes, _stream(stream)))


def mx_glu(z, z_dtype, ldz, live, rows, cols, act, h, h_dtype, ldh, kept_codes=None, kept_ld=0, kept_scales=None,
           kept_scale_ld=0, stream=None):
    _check("mx_glu", lib().mx_glu(_ptr(z), z_dtype, ldz, _ptr(live), rows, cols, act, _ptr(h), h_dtype, ldh,
                                  _ptr(kept_codes), kept_ld, _ptr(kept_scales), kept_scale_ld, _stream(stream)))


def mx_glu_quantize(z, z_dtype, ldz, live, rows, cols, act, codes, scales, scale_ld, kept_codes=None, kept_ld=0,
                    kept_scales=None, kept_scale_ld=0, stream=None):
    _check("mx_glu_quantize", lib().mx_glu_quantize(
        _ptr(z), z_dtype, ldz, _ptr(live), rows, cols, act, _ptr(codes), _ptr(scales), scale_ld,
        _ptr(kept_codes), kept_ld, _ptr(kept_scales), kept_scale_ld, _stream(stream)))


def mx_glu_quantize8(z, z_dtype, ldz, live, rows, cols, act, codes, ld, scales, scale_ld, kept_codes=None,
                     kept_ld=0, kept_scales=None, kept_scale_ld=0, stream=None):
    _check("mx_glu_quantize8", lib().mx_glu_quantize8(
        _ptr(z), z_dtype, ldz, _ptr(live), rows, cols, act, _ptr(codes), ld, _ptr(scales), scale_ld,
        _ptr(kept_codes), kept_ld, _ptr(kept_scales), kept_scale_ld, _stream(stream)))


def mx_glu_bwd(dh, dh_dtype, lddh, kept_codes, kept_ld, kept_scales, kept_scale_ld, live, rows, cols, act, dz,
               dz_dtype, lddz, stream=None):
    _check("mx_glu_bwd", lib().mx_glu_bwd(
        _ptr(dh), dh_dtype, lddh, _ptr(kept_codes), kept_ld, _ptr(kept_scales), kept_scale_ld, _ptr(live), rows,
        cols, act, _ptr(dz), dz_dtype, lddz, _stream(stream)))


def mx_moe_route_workspace_size(tokens, experts, top_k) -> int:
    return int(lib().mx_moe_route_workspace_size(tokens, experts, top_k))


def mx_moe_route(logits, dtype, ld, mask, tokens, experts, top_k, renormalize, ids, weights, counts, sums, loss,
                 workspace=None, workspace_bytes=0, stream=None):
    _check("mx_moe_route", lib().mx_moe_route(
        _ptr(logits), dtype, ld, _ptr(mask), tokens, experts, top_k, renormalize, _ptr(ids), _ptr(weights),
        _ptr(counts), _ptr(sums), _ptr(loss), _ptr(workspace), workspace_bytes, _stream(stream)))


def mx_moe_route_bwd(logits, dtype, ld, mask, tokens, experts, top_k, renormalize, ids, counts, dweights, dloss,
                     dlogits, ldd, stream=None):
    _check("mx_moe_route_bwd", lib().mx_moe_route_bwd(
        _ptr(logits), dtype, ld, _ptr(mask), tokens, experts, top_k, renormalize, _ptr(ids), _ptr(counts),
        _ptr(dweights), _ptr(dloss), _ptr(dlogits), ldd, _stream(stream)))


def mx_deosc_init(w, rows, cols, w_prev, d_w, d_q, stream=None):
    _check("mx_deosc_init", lib().mx_deosc_init(_ptr(w), rows, cols, _ptr(w_prev), _ptr(d_w),
                                                _ptr(d_q), _stream(stream)))


def mx_deosc_step(w, rows, cols, w_prev, d_w, d_q, end_of_window, threshold, flags, stream=None):
    _check("mx_deosc_step", lib().mx_deosc_step(_ptr(w), rows, cols, _ptr(w_prev), _ptr(d_w),
                                                _ptr(d_q), int(end_of_window), threshold,
                                                _ptr(flags), _stream(stream)))


def mx_deosc_step_quantize(w, rows, cols, w_prev, d_w, d_q, end_of_window, threshold, flags,
                           wq_codes, wq_scales, stream=None):
    _check("mx_deosc_step_quantize",
           lib().mx_deosc_step_quantize(_ptr(w), rows, cols, _ptr(w_prev), _ptr(d_w), _ptr(d_q),
                                        int(end_of_window), threshold, _ptr(flags),
                                        _ptr(wq_codes), _ptr(wq_scales), _stream(stream)))


def mx_qema_step(w, ema, rows, cols, beta, wq_codes, wq_scales, stream=None):
    _check("mx_qema_step", lib().mx_qema_step(_ptr(w), _ptr(ema), rows, cols, beta,
                                              _ptr(wq_codes), _ptr(wq_scales), _stream(stream)))


def mx_synth_step(w, n, seed, step, stream=None):
    _check("mx_synth_step", synth_lib().mx_synth_step(_ptr(w), n, seed, step, _stream(stream)))


# ------------------------------------------------------------------ tensor conveniences
def _u8(shape, device):
    return torch.empty(shape, dtype=torch.uint8, device=device)


def quantize(x: torch.Tensor, axis=MX_ROW, round=MX_RNE, seed=0, hadamard=False, sign_mask=0,
             stream=None):
    """Packed (codes, scales) of a 2-D float32/bf16 device tensor."""
    rows, cols = x.shape
    outer, inner = (rows, cols) if axis == MX_ROW else (cols, rows)
    codes = _u8((outer, inner // 2), x.device)
    scales = _u8((outer, inner // 32), x.device)
    mx_quantize(x, dtype_code(x), rows, cols, axis, round, seed, int(bool(hadamard)), sign_mask,
                codes, scales, stream)
    return codes, scales


def dequantize(codes, scales, rows, cols, axis=MX_ROW, hadamard=False, sign_mask=0,
               out_dtype=torch.float32, stream=None):
    out = torch.empty((rows, cols), dtype=out_dtype, device=codes.device)
    mx_dequantize(codes, scales, rows, cols, axis, int(bool(hadamard)), sign_mask, out,
                  dtype_code(out), stream)
    return out


def requantize(codes, scales, rows, cols, round=MX_SR, seed=0, stream=None):
    co = _u8((cols, rows // 2), codes.device)
    so = _u8((cols, rows // 32), codes.device)
    mx_requantize(codes, scales, rows, cols, round, seed, co, so, stream)
    return co, so


def gemm(a, b, M, N, K, alpha=1.0, stream=None):
    c = torch.empty((M, N), dtype=torch.float32, device=a[0].device)
    mx_gemm(a[0], a[1], b[0], b[1], M, N, K, alpha, c, N, stream)
    return c


def linear_fwd(x: torch.Tensor, w: torch.Tensor, stream=None):
    M, K = x.shape
    N = w.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    xq = (_u8((M, K // 2), x.device), _u8((M, K // 32), x.device))
    wq = (_u8((N, K // 2), x.device), _u8((N, K // 32), x.device))
    mx_linear_fwd(x, w, dtype_code(x), M, N, K, y, xq[0], xq[1], wq[0], wq[1], stream)
    return y, xq, wq


def linear_fwd_rht(x: torch.Tensor, w: torch.Tensor, sign_mask: int, stream=None):
    M, K = x.shape
    N = w.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    xq = (_u8((M, K // 2), x.device), _u8((M, K // 32), x.device))
    wq = (_u8((N, K // 2), x.device), _u8((N, K // 32), x.device))
    mx_linear_fwd_rht(x, w, dtype_code(x), M, N, K, sign_mask, y, xq[0], xq[1], wq[0], wq[1],
                      stream)
    return y, xq, wq


def linear_bwd_rht(dy: torch.Tensor, xq, wq, M, N, K, seed, sign_mask, workspace=None,
                   stream=None):
    need = mx_linear_bwd_workspace_size(M, N, K)
    if workspace is None:
        workspace = _u8((need,), dy.device)
    dx = torch.empty((M, K), dtype=torch.float32, device=dy.device)
    dw = torch.empty((N, K), dtype=torch.float32, device=dy.device)
    mx_linear_bwd_rht(dy, dtype_code(dy), M, N, K, xq[0], xq[1], wq[0], wq[1], seed, sign_mask,
                      dx, dw, workspace, workspace.numel(), stream)
    return dx, dw


def grouped_linear_bwd(dy: torch.Tensor, xq, wq, offs, N, K, seed, workspace=None, stream=None):
    """dX [R, K] and dW [groups, N, K] of a grouped layer (offs: host offsets)."""
    G = len(offs) - 1
    R = int(offs[-1])
    need = mx_grouped_linear_bwd_workspace_size(offs, G, N, K)
    if workspace is None:
        workspace = _u8((need,), wq[0].device)
    dx = torch.empty((R, K), dtype=torch.float32, device=wq[0].device)
    dw = torch.empty((G, N, K), dtype=torch.float32, device=wq[0].device)
    mx_grouped_linear_bwd(dy, dtype_code(dy), offs, G, N, K, xq[0], xq[1], wq[0], wq[1], seed, dx,
                          dw, workspace, workspace.numel(), stream)
    return dx, dw


def linear_bwd(dy: torch.Tensor, xq, wq, M, N, K, seed, workspace=None, stream=None):
    need = mx_linear_bwd_workspace_size(M, N, K)
    if workspace is None:
        workspace = _u8((need,), dy.device)
    dx = torch.empty((M, K), dtype=torch.float32, device=dy.device)
    dw = torch.empty((N, K), dtype=torch.float32, device=dy.device)
    mx_linear_bwd(dy, dtype_code(dy), M, N, K, xq[0], xq[1], wq[0], wq[1], seed, dx, dw,
                  workspace, workspace.numel(), stream)
    return dx, dw


# The conveniences below check what the C calls cannot see: types, shapes, that
# every tensor and the stream are the current device's and that rows are contiguous
# (row strides are passed on).  Outputs are allocated on the stream the call runs on.  They sit
# in front of calls of a few microseconds, so the checks are plain conditions and
# messages are made only for an error.
def _device_error(tensors):
    bad = [str(t.device) for t in tensors if t is not None and t.get_device() != torch.cuda.current_device()]
    return ValueError(f"tensor on {bad[0]}, the current device is cuda:{torch.cuda.current_device()}")


def _on_current_device(*tensors) -> None:
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise _device_error(tensors)


def _row_ld(t: torch.Tensor, what: str) -> int:
    """Row stride in elements of a 2-D tensor with contiguous rows."""
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what}: rows must be contiguous")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{what}: rows must not overlap")
    return ld


def _torch_stream(stream):
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream)
    if stream.device.index != torch._C._cuda_getDevice():
        raise ValueError(f"stream of {stream.device}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return stream


def _empty(shape, dtype, like, stream):
    """A tensor of the current device, allocated on the stream the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(_torch_stream(stream)):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _keep(stream, *tensors) -> None:
    """Keeps the memory of tensors from reuse until the given stream is done with them."""
    if stream is not None:
        stream = _torch_stream(stream)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _output(out, shape, dtype, like, stream):
    if out is None:
        return _empty(shape, dtype, like, stream)
    if out.shape != shape or out.dtype != dtype:
        raise ValueError(f"out must be {tuple(shape)} {dtype}, not {tuple(out.shape)} {out.dtype}")
    return out


def _check_workspace(workspace) -> None:
    """The library takes a workspace as one run of bytes."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _workspace(workspace, need, like, stream):
    return _empty((need,), torch.uint8, like, stream) if workspace is None and need else workspace


def _nbytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _check_packed(codes, scales, K):
    """Leading dimensions of packed weights and the pitch of their scale rows."""
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError("packed weights are uint8")
    *rows, half = codes.shape
    *scale_rows, scale_ld = scales.shape
    if rows != scale_rows:
        raise ValueError("codes and scales must have the same rows")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("packed weights must be contiguous")
    if 2 * half != K:
        raise ValueError(f"x has {K} columns, the weight {2 * half}")
    return rows, scale_ld


def gemv(x: torch.Tensor, w, alpha=1.0, out=None, out_dtype=torch.float32, workspace=None,
         stream=None):
    """alpha x deq(W)^T of a few rows x [M, K] (float32 or bf16) and a packed weight
    w = (codes [N, K/2], scales [N, >= K/32]); returns [M, N]."""
    codes, scales = w
    M, K = x.shape
    rows, scale_ld = _check_packed(codes, scales, K)
    if len(rows) != 1:
        raise ValueError("one packed weight has codes [N, K/2] and scales [N, >= K/32]")
    N = rows[0]
    _check_workspace(workspace)
    _on_current_device(x, codes, scales, out, workspace)
    xt, ldx = dtype_code(x), _row_ld(x, "x")
    if out is not None:
        out_dtype = out.dtype
    y = _output(out, (M, N), out_dtype, x, stream)
    _keep(stream, x, codes, scales, out, workspace)
    workspace = _workspace(workspace, mx_gemv_workspace_size(xt, M, N, K), x, stream)
    mx_gemv(x, xt, ldx, codes, scales, scale_ld, M, N, K, alpha, y, dtype_code(y),
            _row_ld(y, "out"), workspace, _nbytes(workspace), stream)
    return y


def gemv_grouped(x: torch.Tensor, w, offs, src=None, top_k=1, alpha=1.0, out=None,
                 out_dtype=torch.float32, stream=None):
    """Each routed row's alpha x deq(W_e)^T, offsets on the device (moe_plan's offs and
    src): w = (codes [E, N, K/2], scales [E, N, >= K/32]); returns [rows, N], where rows
    is src's length (without src: x's rows, each its own).  Rows from offs[E] on are
    left as `out` had them."""
    codes, scales = w
    xr, K = x.shape
    groups = offs.numel() - 1
    w_rows, scale_ld = _check_packed(codes, scales, K)
    if len(w_rows) != 2 or w_rows[0] != groups:
        raise ValueError(f"codes and scales must have the same rows, {groups} groups of them")
    N = w_rows[1]
    if offs.dtype != torch.int64 or not offs.is_contiguous():
        raise ValueError("offs must be int64")
    if src is not None and (src.dtype != torch.int32 or not src.is_contiguous()):
        raise ValueError("src must be int32")
    _on_current_device(x, codes, scales, offs, src, out)
    rows = xr if src is None else src.numel()
    if out is not None:
        out_dtype = out.dtype
    y = _output(out, (rows, N), out_dtype, x, stream)
    _keep(stream, x, codes, scales, offs, src, out)
    mx_gemv_grouped(x, dtype_code(x), _row_ld(x, "x"), xr, src, top_k, codes, scales, scale_ld,
                    offs, groups, rows, N, K, alpha, y, dtype_code(y), _row_ld(y, "out"), stream)
    return y


def moe_plan(ids: torch.Tensor, experts: int, workspace=None, stream=None):
    """(offs [experts + 1] int64, src [tokens * top_k] int32, pos [tokens, top_k] int32) of
    the expert ids [tokens, top_k] (int32 or int64; out of range: the slot is left out)."""
    tokens, top_k = ids.shape
    wide = ids.dtype == torch.int64
    if not wide and ids.dtype != torch.int32:
        raise ValueError("ids must be int32 or int64")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    _check_workspace(workspace)
    _on_current_device(ids, workspace)
    _keep(stream, ids, workspace)
    workspace = _workspace(workspace, mx_moe_plan_workspace_size(tokens, top_k, experts), ids, stream)
    offs = _empty((experts + 1,), torch.int64, ids, stream)
    src = _empty((tokens * top_k,), torch.int32, ids, stream)
    pos = _empty((tokens, top_k), torch.int32, ids, stream)
    mx_moe_plan(ids, MX_I64 if wide else MX_I32, tokens, top_k, experts, offs, src, pos, workspace,
                _nbytes(workspace), stream)
    return offs, src, pos


def _routing(pos, weights, tokens):
    """top_k of pos [tokens, top_k]."""
    if pos.dim() != 2 or pos.dtype != torch.int32 or not pos.is_contiguous():
        raise ValueError("pos must be int32 [tokens, top_k]")
    if pos.shape[0] != tokens:
        raise ValueError(f"pos is for {pos.shape[0]} tokens, not {tokens}")
    if weights is not None and (weights.dtype != torch.float32 or weights.shape != pos.shape
                                or not weights.is_contiguous()):
        raise ValueError("weights must be float32 like pos")
    return pos.shape[1]


def _check_rows(rows, out_rows) -> None:
    if rows is not None and rows != out_rows:
        raise ValueError(f"out has {out_rows} rows, not {rows}")


def moe_dispatch(x: torch.Tensor, pos, weights=None, rows=None, out=None, stream=None):
    """Rows of x [tokens, cols] copied (times weights) to out[pos]: [rows, cols], rows = all
    slots if neither it nor out is given.  Rows no slot maps to are left as `out` had them."""
    tokens, cols = x.shape
    top_k = _routing(pos, weights, tokens)
    if out is not None:
        _check_rows(rows, out.shape[0])
        rows = out.shape[0]
    elif rows is None:
        rows = pos.numel()
    _on_current_device(x, pos, weights, out)
    o = _output(out, (rows, cols), x.dtype, x, stream)
    _keep(stream, x, pos, weights, out)
    mx_moe_dispatch(x, dtype_code(x), _row_ld(x, "x"), pos, weights, tokens, top_k, rows, cols, o,
                    _row_ld(o, "out"), stream)
    return o


def moe_dispatch_quantize(x: torch.Tensor, pos, rows=None, out=None, stream=None):
    """Packed (codes [rows, cols/2], scales [rows, >= cols/32]) of moe_dispatch(x, pos); the
    scale row pitch is that of out's scales, cols/32 if out is not given."""
    tokens, cols = x.shape
    top_k = _routing(pos, None, tokens)
    if out is None:
        rows = pos.numel() if rows is None else rows
        out = (_empty((rows, cols // 2), torch.uint8, x, stream),
               _empty((rows, cols // 32), torch.uint8, x, stream))
    codes, scales = out
    _check_rows(rows, codes.shape[0])
    rows = codes.shape[0]
    if (codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous()
            or not scales.is_contiguous() or codes.dim() != 2 or codes.shape[1] != cols // 2
            or scales.dim() != 2 or scales.shape[0] != rows):
        raise ValueError("out must be packed uint8 codes and scales")
    _on_current_device(x, pos, codes, scales)
    _keep(stream, x, pos, codes, scales)
    mx_moe_dispatch_quantize(x, dtype_code(x), _row_ld(x, "x"), pos, tokens, top_k, rows, cols, codes,
                             scales, scales.shape[1], stream)
    return codes, scales


def moe_combine(z: torch.Tensor, pos, weights=None, out=None, out_dtype=torch.float32, stream=None):
    """y[t] = sum_j weights[t, j] z[pos[t, j]] [tokens, cols]; without weights the gradient of
    moe_dispatch."""
    rows, cols = z.shape
    tokens = pos.shape[0]
    top_k = _routing(pos, weights, tokens)
    _on_current_device(z, pos, weights, out)
    if out is not None:
        out_dtype = out.dtype
    y = _output(out, (tokens, cols), out_dtype, z, stream)
    _keep(stream, z, pos, weights, out)
    mx_moe_combine(z, dtype_code(z), _row_ld(z, "z"), rows, pos, weights, tokens, top_k, cols, y,
                   dtype_code(y), _row_ld(y, "out"), stream)
    return y


def moe_combine_bwd(dy: torch.Tensor, z: torch.Tensor, pos, weights=None, out=None, stream=None):
    """(dz [rows, cols] of dy's type, dweights [tokens, top_k] float32) of moe_combine(z, pos,
    weights); dz's rows that no slot maps to are left as `out` had them."""
    tokens, cols = dy.shape
    rows = z.shape[0]
    top_k = _routing(pos, weights, tokens)
    if z.dim() != 2 or z.shape[1] != cols:
        raise ValueError("z and dy must have the same columns")
    _on_current_device(dy, z, pos, weights, out)
    dz = _output(out, (rows, cols), dy.dtype, dy, stream)
    _keep(stream, dy, z, pos, weights, out)
    dw = _empty((tokens, top_k), torch.float32, dy, stream)
    mx_moe_combine_bwd(dy, dtype_code(dy), _row_ld(dy, "dy"), z, dtype_code(z), _row_ld(z, "z"), rows,
                       pos, weights, tokens, top_k, cols, dz, _row_ld(dz, "out"), dw, stream)
    return dz, dw


# ------------------------------------------------------------------ 8-bit matrices
def _matrix8(rows, cols, like, stream):
    """An 8-bit matrix [rows, cols] to write: codes [rows, cols rounded up to 16], scales
    [rows, 4 bytes per 512 columns]."""
    return (_empty((rows, -(-cols // 16) * 16), torch.uint8, like, stream),
            _empty((rows, -(-cols // 512) * 4), torch.uint8, like, stream))


def _check_matrix8(m, what: str, cols=None):
    """(rows, code pitch, scale pitch) of an 8-bit matrix of `cols` columns (None: its codes')."""
    codes, scales = m
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError(f"{what}: codes and scales are uint8")
    shape, blocks = codes.shape, scales.shape
    if len(shape) != 2 or len(blocks) != 2 or shape[0] != blocks[0]:
        raise ValueError(f"{what}: codes [rows, cols] and scales [rows, blocks] must have the same rows")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{what}: codes and scales must be contiguous")
    (rows, ld), scale_ld = shape, blocks[1]
    cols = ld if cols is None else cols
    if ld % 16 or ld < cols or scale_ld % 4 or scale_ld * 128 < cols:
        raise ValueError(f"{what}: rows of {ld} codes and {scale_ld} scales do not hold {cols} columns")
    return rows, ld, scale_ld


def quantize8(x: torch.Tensor, axis=MX_ROW, stream=None):
    """The 8-bit matrix (codes, scales) of x [rows, cols] (float32 or bf16) in 1x128 blocks, or of
    its transpose in 128x1 blocks (MX_COL)."""
    rows, cols = x.shape
    ldx = _row_ld(x, "x")
    _on_current_device(x)
    q = _matrix8(rows, cols, x, stream) if axis == MX_ROW else _matrix8(cols, rows, x, stream)
    _keep(stream, x)
    mx_quantize8(x, dtype_code(x), ldx, rows, cols, axis, q[0], q[0].shape[1], q[1], q[1].shape[1], stream)
    return q


def quantize8_dual(x: torch.Tensor, tile=False, stream=None):
    """(codes, scales, codes_t, scales_t) of x [rows, cols] from one read: x in 1x128 and its transpose
    in 128x1 blocks, or both in the same 128x128 tiles (a weight)."""
    rows, cols = x.shape
    ldx = _row_ld(x, "x")
    _on_current_device(x)
    q, t = _matrix8(rows, cols, x, stream), _matrix8(cols, rows, x, stream)
    _keep(stream, x)
    mx_quantize8_dual(x, dtype_code(x), ldx, rows, cols, int(bool(tile)), q[0], q[0].shape[1], q[1], q[1].shape[1],
                      t[0], t[0].shape[1], t[1], t[1].shape[1], stream)
    return (*q, *t)


def requantize8(q, cols=None, stream=None):
    """The transpose of an 8-bit matrix [rows, cols] (cols: its code row's length by default), its
    values quantized again in 128x1 blocks."""
    rows, ld, scale_ld = _check_matrix8(q, "q", cols)
    cols = ld if cols is None else cols
    _on_current_device(*q)
    t = _matrix8(cols, rows, q[0], stream)
    _keep(stream, *q)
    mx_requantize8(q[0], ld, q[1], scale_ld, rows, cols, t[0], t[0].shape[1], t[1], t[1].shape[1], stream)
    return t


def dequantize8(q, cols=None, out_dtype=torch.float32, stream=None):
    """The values [rows, cols] of an 8-bit matrix (cols: its code row's length by default)."""
    rows, ld, scale_ld = _check_matrix8(q, "q", cols)
    cols = ld if cols is None else cols
    _on_current_device(*q)
    out = _empty((rows, cols), out_dtype, q[0], stream)
    _keep(stream, *q)
    mx_dequantize8(q[0], ld, q[1], scale_ld, rows, cols, out, dtype_code(out), cols, stream)
    return out


def gemm8(a, b, alpha=1.0, out=None, out_dtype=torch.float32, workspace=None, stream=None):
    """alpha A B^T [M, N] of two 8-bit matrices (codes, scales), A [M, K] and B [N, K].  A float32 result
    sums exact products; a bf16 one takes the 8-bit matrix instructions, which add eight neighbouring products
    with 13 bits below the largest (2^-10 of their magnitudes at most, 2e-5 of the result's norm on normal
    operands): where large terms cancel, ask for float32."""
    M, lda, lsa = _check_matrix8(a, "a")
    N, ldb, lsb = _check_matrix8(b, "b")
    if lda != ldb:
        raise ValueError(f"a has rows of {lda} codes, b of {ldb}")
    _check_workspace(workspace)
    _on_current_device(*a, *b, out, workspace)
    if out is not None:
        out_dtype = out.dtype
    c = _output(out, (M, N), out_dtype, a[0], stream)
    _keep(stream, *a, *b, out, workspace)
    workspace = _workspace(workspace, mx_gemm8_workspace_size(M, N, lda), a[0], stream)
    mx_gemm8(a[0], lda, a[1], lsa, b[0], ldb, b[1], lsb, M, N, lda, alpha, c, dtype_code(c), _row_ld(c, "out"),
             workspace, _nbytes(workspace), stream)
    return c


def _check_exact8(m, what: str, rows: int, cols: int) -> None:
    """An 8-bit matrix of just this size, as _matrix8 lays it out."""
    r, ld, scale_ld = _check_matrix8(m, what, cols)
    if r != rows or ld != -(-cols // 16) * 16 or scale_ld != -(-cols // 512) * 4:
        raise ValueError(f"{what} is not the 8-bit matrix of [{rows}, {cols}]")


def linear8_fwd(x: torch.Tensor, w, out=None, out_dtype=torch.float32, backward=True, workspace=None, stream=None):
    """(y, xq, wq) of the 8-bit linear layer: y = Q(x) Q(w)^T [M, N] of x [M, K] and w [N, K] (float32 or
    bf16), xq the 8-bit checkpoint of x, wq = (codes, scales, codes_t, scales_t) the weight's tiles in both
    layouts (the first alone without `backward`).  w may be such a wq of an earlier call.  A bf16 y is summed
    as a bf16 gemm8."""
    M, K = x.shape
    quantized = not isinstance(w, torch.Tensor)
    if quantized:
        if len(w) not in (2, 4):
            raise ValueError("a quantized weight is (codes, scales) or (codes, scales, codes_t, scales_t)")
        N = w[0].shape[0]
        _check_exact8(w[:2], "w", N, K)
        wq, ldw, wt = tuple(w), K, MX_F32
    else:
        N = w.shape[0]
        if w.dim() != 2 or w.shape[1] != K:
            raise ValueError(f"x has {K} columns, the weight {tuple(w.shape)}")
        ldw, wt = _row_ld(w, "w"), dtype_code(w)
    _check_workspace(workspace)
    _on_current_device(x, *(w if quantized else (w,)), out, workspace)
    xt, ldx = dtype_code(x), _row_ld(x, "x")
    if out is not None:
        out_dtype = out.dtype
    y = _output(out, (M, N), out_dtype, x, stream)
    yt, ldy = dtype_code(y), _row_ld(y, "out")
    xq = _matrix8(M, K, x, stream)
    if not quantized:
        wq = _matrix8(N, K, x, stream) + (_matrix8(K, N, x, stream) if backward else ())
    _keep(stream, x, *(w if quantized else (w,)), out, workspace)
    workspace = _workspace(workspace, mx_linear8_fwd_workspace_size(M, N, K), x, stream)
    t = wq[2:] if len(wq) == 4 else (None, None)
    mx_linear8_fwd(x, xt, ldx, None if quantized else w, wt, ldw, M, N, K, y, yt, ldy, *xq, *wq[:2], *t, workspace,
                   _nbytes(workspace), stream)
    return y, xq, wq


def linear8_bwd(dy: torch.Tensor, xq, wq, M, N, K, dx_dtype=torch.float32, workspace=None, stream=None):
    """(dx [M, K] of dx_dtype, dw [N, K] float32) of linear8_fwd, given dy [M, N] and what it kept.  A bf16 dx is
    summed as a bf16 gemm8."""
    if tuple(dy.shape) != (M, N):
        raise ValueError(f"dy must be [{M}, {N}], not {tuple(dy.shape)}")
    if len(wq) != 4:
        raise ValueError("the backward takes the weight in both layouts (linear8_fwd with backward=True)")
    _check_exact8(xq, "xq", M, K)
    _check_exact8(wq[2:], "wq", K, N)
    _check_workspace(workspace)
    _on_current_device(dy, *xq, *wq, workspace)
    dyt, lddy = dtype_code(dy), _row_ld(dy, "dy")
    dx = _empty((M, K), dx_dtype, dy, stream)
    dw = _empty((N, K), torch.float32, dy, stream)
    _keep(stream, dy, *xq, *wq, workspace)
    workspace = _workspace(workspace, mx_linear8_bwd_workspace_size(M, N, K), dy, stream)
    mx_linear8_bwd(dy, dyt, lddy, M, N, K, *xq, *wq[2:], dx, dtype_code(dx), K, dw, K, workspace, _nbytes(workspace),
                   stream)
    return dx, dw


# ------------------------------------------------------------------ gated activation
def _glu_rows(rows) -> None:
    if rows is not None and (not isinstance(rows, torch.Tensor) or rows.dtype != torch.int64 or rows.numel() != 1):
        raise ValueError("rows must be one int64 on the device (moe_plan's offs[-1:])")


def _glu_kept(rows, cols, like, stream):
    return _matrix8(2 * rows, cols, like, stream)


def _glu_size(z):
    if z.dim() != 2 or z.shape[1] % 2:
        raise ValueError("z must be [rows, 2 cols]")
    return z.shape[0], z.shape[1] // 2


def glu(z: torch.Tensor, act=MX_SILU, rows=None, checkpoint=False, out=None, out_dtype=torch.float32, stream=None):
    """h = act(g) u [rows, cols] of z = (g, u) [rows, 2 cols]; with checkpoint (h, kept), kept the 8-bit matrix
    of z's halves [2 rows, cols] that glu_bwd takes.  rows: device counter of the rows in use (moe_plan's
    offs[-1:]); those behind are left as `out` had them."""
    n, cols = _glu_size(z)
    _glu_rows(rows)
    _on_current_device(z, rows, out)
    zt, ldz = dtype_code(z), _row_ld(z, "z")
    if out is not None:
        out_dtype = out.dtype
    h = _output(out, (n, cols), out_dtype, z, stream)
    ht, ldh = dtype_code(h), _row_ld(h, "out")
    kept = _glu_kept(n, cols, z, stream) if checkpoint else None
    _keep(stream, z, rows, out)
    k = (kept[0], kept[0].shape[1], kept[1], kept[1].shape[1]) if checkpoint else (None, 0, None, 0)
    mx_glu(z, zt, ldz, rows, n, cols, act, h, ht, ldh, *k, stream)
    return (h, kept) if checkpoint else h


def glu_quantize(z: torch.Tensor, act=MX_SILU, rows=None, checkpoint=False, out=None, stream=None):
    """glu with h as packed MXFP4 (codes [rows, cols/2], scales [rows, >= cols/32]), the operand of the
    next product."""
    n, cols = _glu_size(z)
    _glu_rows(rows)
    if out is None:
        out = _empty((n, cols // 2), torch.uint8, z, stream), _empty((n, cols // 32), torch.uint8, z, stream)
    codes, scales = out
    if (codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not codes.is_contiguous()
            or not scales.is_contiguous() or codes.shape != (n, cols // 2) or scales.dim() != 2
            or scales.shape[0] != n):
        raise ValueError("out must be packed uint8 codes and scales")
    _on_current_device(z, rows, codes, scales)
    zt, ldz = dtype_code(z), _row_ld(z, "z")
    kept = _glu_kept(n, cols, z, stream) if checkpoint else None
    _keep(stream, z, rows, codes, scales)
    k = (kept[0], kept[0].shape[1], kept[1], kept[1].shape[1]) if checkpoint else (None, 0, None, 0)
    mx_glu_quantize(z, zt, ldz, rows, n, cols, act, codes, scales, scales.shape[1], *k, stream)
    return ((codes, scales), kept) if checkpoint else (codes, scales)


def glu_quantize8(z: torch.Tensor, act=MX_SILU, rows=None, checkpoint=False, out=None, stream=None):
    """glu with h as an 8-bit matrix (codes, scales), gemm8's operand."""
    n, cols = _glu_size(z)
    _glu_rows(rows)
    q = _matrix8(n, cols, z, stream) if out is None else out
    r, ld, scale_ld = _check_matrix8(q, "out", cols)
    if r != n:
        raise ValueError(f"out has {r} rows, not {n}")
    _on_current_device(z, rows, *q)
    zt, ldz = dtype_code(z), _row_ld(z, "z")
    kept = _glu_kept(n, cols, z, stream) if checkpoint else None
    _keep(stream, z, rows, *q)
    k = (kept[0], kept[0].shape[1], kept[1], kept[1].shape[1]) if checkpoint else (None, 0, None, 0)
    mx_glu_quantize8(z, zt, ldz, rows, n, cols, act, q[0], ld, q[1], scale_ld, *k, stream)
    return (tuple(q), kept) if checkpoint else tuple(q)


def glu_bwd(dh: torch.Tensor, kept, act=MX_SILU, rows=None, out=None, out_dtype=None, stream=None):
    """dz [rows, 2 cols] (of dh's type by default) of glu, given dh [rows, cols] and the checkpoint; rows behind
    the counter `rows` are left as `out` had them."""
    n, cols = dh.shape
    r, ld, scale_ld = _check_matrix8(kept, "kept", cols)
    if r != 2 * n:
        raise ValueError(f"kept has {r} rows, not {2 * n}")
    _glu_rows(rows)
    _on_current_device(dh, *kept, rows, out)
    dt, lddh = dtype_code(dh), _row_ld(dh, "dh")
    dz = _output(out, (n, 2 * cols), out.dtype if out is not None else out_dtype or dh.dtype, dh, stream)
    _keep(stream, dh, *kept, rows, out)
    mx_glu_bwd(dh, dt, lddh, kept[0], ld, kept[1], scale_ld, rows, n, cols, act, dz, dtype_code(dz),
               _row_ld(dz, "out"), stream)
    return dz


# ------------------------------------------------------------------ router
def _route_mask(mask, tokens) -> None:
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (tokens,)
                             or not mask.is_contiguous()):
        raise ValueError("mask must be bool [tokens]")


def moe_route(logits: torch.Tensor, top_k: int, renormalize=True, mask=None, workspace=None, stream=None):
    """(ids [tokens, top_k] int32, weights [tokens, top_k] float32, counts [experts + 1] int32, sums [experts]
    float32, loss [1] float32) of router logits [tokens, experts]: each token's top_k experts (-1: slot left
    out, moe_plan's convention) and their softmax weights, slots per expert and behind them the tokens that take
    part, the softmax's sums over those, and the balance loss.  mask [tokens]: False for padding tokens."""
    tokens, experts = logits.shape
    _route_mask(mask, tokens)
    _check_workspace(workspace)
    _on_current_device(logits, mask, workspace)
    lt, ld = dtype_code(logits), _row_ld(logits, "logits")
    _keep(stream, logits, mask, workspace)
    workspace = _workspace(workspace, mx_moe_route_workspace_size(tokens, experts, top_k), logits, stream)
    ids = _empty((tokens, top_k), torch.int32, logits, stream)
    weights = _empty((tokens, top_k), torch.float32, logits, stream)
    counts = _empty((experts + 1,), torch.int32, logits, stream)
    sums = _empty((experts,), torch.float32, logits, stream)
    loss = _empty((1,), torch.float32, logits, stream)
    mx_moe_route(logits, lt, ld, mask, tokens, experts, top_k, int(bool(renormalize)), ids, weights, counts, sums,
                 loss, workspace, _nbytes(workspace), stream)
    return ids, weights, counts, sums, loss


def moe_route_bwd(logits: torch.Tensor, ids, counts, dweights=None, dloss=None, renormalize=True, mask=None,
                  out=None, stream=None):
    """dlogits [tokens, experts] (logits' type) of moe_route, given its ids and counts and the gradients of its
    weights (moe_combine_bwd's dweights) and of its loss ([1] float32), each None for 0."""
    tokens, experts = logits.shape
    _route_mask(mask, tokens)
    if ids.dtype != torch.int32 or ids.dim() != 2 or ids.shape[0] != tokens or not ids.is_contiguous():
        raise ValueError("ids must be int32 [tokens, top_k]")
    if counts.dtype != torch.int32 or counts.shape != (experts + 1,) or not counts.is_contiguous():
        raise ValueError("counts must be int32 [experts + 1]")
    if dweights is not None and (dweights.dtype != torch.float32 or dweights.shape != ids.shape
                                 or not dweights.is_contiguous()):
        raise ValueError("dweights must be float32 like ids")
    if dloss is not None and (dloss.dtype != torch.float32 or dloss.numel() != 1):
        raise ValueError("dloss must be one float32")
    _on_current_device(logits, ids, counts, dweights, dloss, mask, out)
    lt, ld = dtype_code(logits), _row_ld(logits, "logits")
    d = _output(out, (tokens, experts), logits.dtype, logits, stream)
    _keep(stream, logits, ids, counts, dweights, dloss, mask, out)
    mx_moe_route_bwd(logits, lt, ld, mask, tokens, experts, ids.shape[1], int(bool(renormalize)), ids, counts,
                     dweights, dloss, d, _row_ld(d, "out"), stream)
    return d
