"""Thin ctypes binding of libfp8bs.so (include/fp8bs.h).

The functions carry the C names and only marshal arguments: tensor -> device
pointer, sizes, strides, and the current torch stream as the HIP stream.
Every step of the computation runs in the HIP library; if the library is not
built or cannot be loaded, every call raises.  PyTorch provides device memory
and streams only.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8bs.so")
_lock = threading.Lock()
_lib = None

STATUS = {0: "FP8BS_OK", 1: "FP8BS_ERR_NULL", 2: "FP8BS_ERR_SHAPE", 3: "FP8BS_ERR_STRIDE",
          4: "FP8BS_ERR_ALIGN", 5: "FP8BS_ERR_UNSUPPORTED", 6: "FP8BS_ERR_DEVICE"}
AXIS_ROW, AXIS_COL = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
BSCALE_BLOCK128, BSCALE_ROW128 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1

EXPORTS = ["fp8_quant_rowblock", "fp8_quant_block2d", "fp8_quant_linear", "fp8_quant_rowwise", "fp8_quant_tensorwise", "fp8_blockscaled_gemm", "fp8_blockscaled_gemm_plan",
           "fp8_blockscaled_gemm_splitk", "fp8_blockscaled_gemm_splitk_noalloc", "fp8_blockscaled_gemm_splitk_plan",
           "fp8_grouped_gemm", "fp8_grouped_gemm_ws_size", "fp8_grouped_gemm_swiglu_quant", "mxfp8_grouped_gemm_swiglu_quant",
           "fp8_silu_mul_quant", "fp8_moe_combine", "fp8_moe_combine_routed", "fp8_moe_combine_backward",
           "fp8_moe_route", "fp8_moe_route_ws_size", "fp8_moe_route_backward",
           "fp8_moe_route_grouped", "fp8_moe_route_grouped_backward", "fp8_moe_bias_update",
           "fp8_block_norm", "fp8_block_norm_backward", "fp8_block_norm_backward_ws_size", "mxfp8_quant", "mxfp8_quant_t",
           "fp8_quant_dual_axis", "fp8_transpose_codes", "fp8_quant_linear_pow2",
           "fp8_quant_pow2", "fp8_blockscaled_gemm_pow2", "mxfp8_gemm", "int8_quant",
           "int8_silu_mul_quant", "int8_gemm", "int8_gemm_ws_size", "int8_linear", "int8_linear_ws_size",
           "int8_linear_backward", "int8_linear_backward_ws_size", "int8_grouped_gemm",
           "fp8bs_e4m3_encode",
           "fp8bs_status_string", "fp8bs_last_error_detail"]


class Fp8bsError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__("%s failed: %s (%s)" % (fn, STATUS.get(status, status), detail))
        self.status = status
        self.detail = detail


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libfp8bs.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libfp8bs.so is not built (%s); run `python -m fp8_block_scaled_x128_amd.build`"
                               % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        P, I64, I32, INT, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
        sig = {
            "fp8_quant_rowblock": [P, I64, I64, I64, INT, P, I64, P, I64, I64, P],
            "fp8_quant_block2d": [P, I64, I64, I64, I64, P, I64, P, I64, P, P],
            "fp8_quant_linear": [P, I64, I64, I64, P, I64, P, I64, I64, P, I64, I64, P, I64, P, P],
            "fp8_quant_rowwise": [P, I64, I64, I64, P, I64, P, P],
            "fp8_quant_tensorwise": [P, I64, I64, I64, P, I64, P, P],
            "fp8_blockscaled_gemm": [I64, I64, I64, P, I64, P, I64, I64, P, I64, P, I64, I64, INT, P, I64, INT, P],
            "fp8_blockscaled_gemm_plan": [I64, I64, I64, P],
            "fp8_blockscaled_gemm_splitk": [I64, I64, I64, P, I64, P, I64, I64, P, I64, P, I64, I64, INT, P, I64,
                                            INT, I32, P, ctypes.c_size_t, P],
            "fp8_blockscaled_gemm_splitk_plan": [I64, I64, I64, INT, P, P],
            "fp8_blockscaled_gemm_splitk_noalloc": [I64, I64, I64, P, I64, P, I64, I64, P, I64, P, I64, I64, INT, P,
                                                    I64, INT, I32, P],
            "fp8_grouped_gemm": [I64, I64, I64, I32, P, P, I64, P, I64, P, I64, I64, P, I64, I64, P, I64, I64, I64,
                                 P, I64, INT, P],
            "fp8_grouped_gemm_ws_size": [I64, I32, I64, P],
            "fp8_grouped_gemm_swiglu_quant": [I64, I64, I64, I32, P, P, I64, P, I64, P, I64, I64, P, I64, I64, P,
                                              I64, I64, I64, P, I64, P, I64, I64, P],
            "mxfp8_grouped_gemm_swiglu_quant": [I64, I64, I64, I32, P, P, I64, P, I64, P, I64, P, I64, I64, P, I64,
                                                I64, P, I64, P, I64, I64, P],
            "fp8_silu_mul_quant": [P, I64, I64, I64, INT, P, I64, P, I64, I64, P, I64, P],
            "fp8_moe_combine": [P, I64, I64, I64, P, P, I64, I32, P, I64, INT, P],
            "fp8_moe_combine_routed": [P, I64, I64, I64, P, P, I64, I32, P, I64, INT, P],
            "fp8_moe_combine_backward": [P, I64, INT, P, I64, I64, I64, P, P, I64, I32, P, I64, P, P],
            "fp8_moe_route": [P, I64, I32, I64, INT, I32, I32, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P],
            "fp8_moe_route_ws_size": [I64, I32, P],
            "fp8_moe_route_backward": [P, I64, I32, I64, INT, I32, I32, P, P, P, P, P, P, P, I64, P],
            "fp8_moe_route_grouped": [P, I64, I32, I64, INT, I32, INT, P, I32, I32, INT, I32, F32, P, P, P, P, P, P, P, P, P,
                                      P, ctypes.c_size_t, P],
            "fp8_moe_route_grouped_backward": [P, I64, I32, I64, INT, I32, INT, I32, F32, P, P, P, P, P, P, I64, P],
            "fp8_moe_bias_update": [P, P, I32, F32, P],
            "fp8_block_norm": [I64, I64, P, I64, P, I64, INT, P, I64, I64, F32, P, P, INT, F32, P, I64, P, I64, P,
                               I64, P, I64, I64, P],
            "fp8_block_norm_backward": [I64, I64, P, I64, INT, P, I64, P, I64, INT, P, I64, P, I64, I64, F32, P, P,
                                        INT, F32, P, I64, P, I64, P, I64, INT, P, P, P, ctypes.c_size_t, P],
            "fp8_block_norm_backward_ws_size": [I64, I64, I64, I32, I32, I32, P],
            "mxfp8_quant": [P, I64, I64, I64, P, I64, P, I64, I64, P],
            "mxfp8_quant_t": [P, I64, I64, I64, P, I64, P, I64, I64, P],
            "fp8_quant_dual_axis": [P, I64, I64, I64, I32, P, I64, P, I64, I64, P, I64, P, I64, I64, P],
            "fp8_transpose_codes": [P, I64, I64, I64, I64, P, I64, P],
            "fp8_quant_linear_pow2": [P, I64, I64, I64, P, I64, P, I64, P, I64, I64, P, I64, P, I64, P],
            "fp8_quant_pow2": [P, I64, I64, I64, I32, P, I64, P, I64, P],
            "fp8_blockscaled_gemm_pow2": [I64, I64, I64, P, I64, P, I64, P, I64, P, I64, P, I64, INT, P],
            "mxfp8_gemm": [I64, I64, I64, I32, P, P, I64, P, I64, P, I64, P, I64, I64, P, I64, I64, P, I64, INT, P],
            "int8_quant": [P, I64, I64, I64, INT, P, I64, P, P],
            "int8_silu_mul_quant": [P, I64, I64, I64, P, P, I64, P, P, I64, P],
            "int8_gemm": [I64, I64, I64, P, I64, P, P, I64, P, P, I64, INT, P, ctypes.c_size_t, P],
            "int8_gemm_ws_size": [I64, I64, I64, P],
            "int8_linear": [I64, I64, I64, P, I64, P, I64, P, P, I64, INT, P, ctypes.c_size_t, P],
            "int8_linear_ws_size": [I64, I64, I64, P],
            "int8_linear_backward": [I64, I64, I64, P, I64, P, I64, P, I64, P, I64, P, I64, P, ctypes.c_size_t, P],
            "int8_linear_backward_ws_size": [I64, I64, I64, P],
            "int8_grouped_gemm": [I64, I64, I64, I32, P, P, I64, P, I64, P, P, I64, I64, P, I64, P, I64, INT, P],
            "fp8bs_e4m3_encode": [P, P, I64, P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.fp8bs_status_string.argtypes = [ctypes.c_int]
        lib.fp8bs_status_string.restype = ctypes.c_char_p
        lib.fp8bs_last_error_detail.argtypes = []
        lib.fp8bs_last_error_detail.restype = ctypes.c_char_p
        _lib = lib
        return lib


# Pointers and streams go to ctypes as plain integers (the argument types are
# c_void_p): building a c_void_p and a torch Stream object per argument cost
# more than the smallest kernels run.
def _p(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name, status, raise_on_error=True):
    if status != 0 and raise_on_error:
        detail = load().fp8bs_last_error_detail().decode()
        raise Fp8bsError(name, status, detail)
    return status


# ---------------------------------------------------------------- raw C calls
def fp8_quant_rowblock(x, rows, cols, ld_x, axis, q, ld_q, s, s_stride_row, s_stride_group, stream=None,
                       raise_on_error=True):
    st = load().fp8_quant_rowblock(_p(x), rows, cols, ld_x, axis, _p(q), ld_q, _p(s), s_stride_row,
                                   s_stride_group, _stream(stream))
    return _check("fp8_quant_rowblock", st, raise_on_error)


def fp8_quant_block2d(w, batch, rows, cols, ld_w, q, ld_q, q_t, ld_qt, s, stream=None, raise_on_error=True):
    st = load().fp8_quant_block2d(_p(w), batch, rows, cols, ld_w, _p(q), ld_q, _p(q_t), ld_qt, _p(s),
                                  _stream(stream))
    return _check("fp8_quant_block2d", st, raise_on_error)


def fp8_quant_linear(x, rows, cols, ld_x, qx, ld_qx, sx, sx_stride_row, sx_stride_group, w, w_rows, ld_w, qw, ld_qw,
                     sw, stream=None, raise_on_error=True):
    st = load().fp8_quant_linear(_p(x), rows, cols, ld_x, _p(qx), ld_qx, _p(sx), sx_stride_row, sx_stride_group,
                                 _p(w), w_rows, ld_w, _p(qw), ld_qw, _p(sw), _stream(stream))
    return _check("fp8_quant_linear", st, raise_on_error)


def fp8_quant_rowwise(x, rows, cols, ld_x, q, ld_q, s, stream=None, raise_on_error=True):
    st = load().fp8_quant_rowwise(_p(x), rows, cols, ld_x, _p(q), ld_q, _p(s), _stream(stream))
    return _check("fp8_quant_rowwise", st, raise_on_error)


def fp8_quant_tensorwise(x, rows, cols, ld_x, q, ld_q, s, stream=None, raise_on_error=True):
    st = load().fp8_quant_tensorwise(_p(x), rows, cols, ld_x, _p(q), ld_q, _p(s), _stream(stream))
    return _check("fp8_quant_tensorwise", st, raise_on_error)


def fp8_blockscaled_gemm(M, N, K, a, lda, sa, sa_stride_m, sa_stride_k, b, ldb, sb, sb_stride_n, sb_stride_k,
                         bscale, c, ldc, out, stream=None, raise_on_error=True):
    st = load().fp8_blockscaled_gemm(M, N, K, _p(a), lda, _p(sa), sa_stride_m, sa_stride_k, _p(b), ldb, _p(sb),
                                     sb_stride_n, sb_stride_k, bscale, _p(c), ldc, out, _stream(stream))
    return _check("fp8_blockscaled_gemm", st, raise_on_error)


def fp8_blockscaled_gemm_plan(M, N, K):
    """Tiling of a BLOCK128 problem: ((waves, weight rows per tile) for columns
    [0, split), (waves, rows) for [split, N) or None, split).  Host only."""
    out = (ctypes.c_int32 * 5)()
    _check("fp8_blockscaled_gemm_plan", load().fp8_blockscaled_gemm_plan(M, N, K, ctypes.cast(out, ctypes.c_void_p)))
    return (out[0], out[1]), ((out[2], out[3]) if out[2] else None), out[4]


def fp8_blockscaled_gemm_splitk(M, N, K, a, lda, sa, sa_stride_m, sa_stride_k, b, ldb, sb, sb_stride_n,
                                sb_stride_k, bscale, c, ldc, out, splits, ws, ws_bytes, stream=None,
                                raise_on_error=True):
    st = load().fp8_blockscaled_gemm_splitk(M, N, K, _p(a), lda, _p(sa), sa_stride_m, sa_stride_k, _p(b), ldb,
                                            _p(sb), sb_stride_n, sb_stride_k, bscale, _p(c), ldc, out, splits,
                                            _p(ws), ws_bytes, _stream(stream))
    return _check("fp8_blockscaled_gemm_splitk", st, raise_on_error)


def fp8_blockscaled_gemm_splitk_noalloc(M, N, K, a, lda, sa, sa_stride_m, sa_stride_k, b, ldb, sb, sb_stride_n,
                                        sb_stride_k, bscale, c, ldc, out, splits, stream=None, raise_on_error=True):
    st = load().fp8_blockscaled_gemm_splitk_noalloc(M, N, K, _p(a), lda, _p(sa), sa_stride_m, sa_stride_k, _p(b),
                                                    ldb, _p(sb), sb_stride_n, sb_stride_k, bscale, _p(c), ldc, out,
                                                    splits, _stream(stream))
    return _check("fp8_blockscaled_gemm_splitk_noalloc", st, raise_on_error)


def fp8_blockscaled_gemm_splitk_plan(M, N, K, out):
    """(splits, workspace bytes) the K-split GEMM chooses.  Host only."""
    sp, wb = ctypes.c_int32(0), ctypes.c_size_t(0)
    _check("fp8_blockscaled_gemm_splitk_plan",
           load().fp8_blockscaled_gemm_splitk_plan(M, N, K, out, ctypes.byref(sp), ctypes.byref(wb)))
    return sp.value, wb.value


def fp8_grouped_gemm_ws_size(max_total_rows, G, N, raise_on_error=True):
    """Workspace bytes of the grouped GEMMs (host only); always 0."""
    out = ctypes.c_size_t(0)
    st = load().fp8_grouped_gemm_ws_size(max_total_rows, G, N, ctypes.byref(out))
    if _check("fp8_grouped_gemm_ws_size", st, raise_on_error) != 0:
        return None
    return out.value


def fp8_grouped_gemm_swiglu_quant(total_rows, I, K, G, offsets, a_rows, a_count, a, lda, sa, sa_stride_m, sa_stride_k,
                                  b, ldb, b_stride_g, sb, sb_stride_g, sb_stride_n, sb_stride_k, hq, ld_hq, hs,
                                  hs_stride_row, hs_stride_group, stream=None, raise_on_error=True):
    st = load().fp8_grouped_gemm_swiglu_quant(total_rows, I, K, G, _p(offsets), _p(a_rows), a_count, _p(a), lda, _p(sa),
                                              sa_stride_m, sa_stride_k, _p(b), ldb, b_stride_g, _p(sb), sb_stride_g,
                                              sb_stride_n, sb_stride_k, _p(hq), ld_hq, _p(hs), hs_stride_row,
                                              hs_stride_group, _stream(stream))
    return _check("fp8_grouped_gemm_swiglu_quant", st, raise_on_error)


def mxfp8_grouped_gemm_swiglu_quant(total_rows, I, K, G, offsets, a_rows, a_count, a, lda, sa, lds_a, b, ldb,
                                    b_stride_g, sb, lds_b, sb_stride_g, hq, ld_hq, hs, hs_stride_row,
                                    hs_stride_group, stream=None, raise_on_error=True):
    st = load().mxfp8_grouped_gemm_swiglu_quant(total_rows, I, K, G, _p(offsets), _p(a_rows), a_count, _p(a), lda,
                                                _p(sa), lds_a, _p(b), ldb, b_stride_g, _p(sb), lds_b, sb_stride_g,
                                                _p(hq), ld_hq, _p(hs), hs_stride_row, hs_stride_group,
                                                _stream(stream))
    return _check("mxfp8_grouped_gemm_swiglu_quant", st, raise_on_error)


def fp8_grouped_gemm(total_rows, N, K, G, offsets, a_rows, a_count, a, lda, sa, sa_stride_m, sa_stride_k, b, ldb,
                     b_stride_g, sb, sb_stride_g, sb_stride_n, sb_stride_k, c, ldc, out, stream=None,
                     raise_on_error=True):
    st = load().fp8_grouped_gemm(total_rows, N, K, G, _p(offsets), _p(a_rows), a_count, _p(a), lda, _p(sa),
                                 sa_stride_m, sa_stride_k, _p(b), ldb, b_stride_g, _p(sb), sb_stride_g, sb_stride_n,
                                 sb_stride_k, _p(c), ldc, out, _stream(stream))
    return _check("fp8_grouped_gemm", st, raise_on_error)


def fp8_silu_mul_quant(gate_up, rows, I, ld_in, mx, q, ld_q, s, s_stride_row, s_stride_group, h_out, ld_h,
                       stream=None, raise_on_error=True):
    st = load().fp8_silu_mul_quant(_p(gate_up), rows, I, ld_in, mx, _p(q), ld_q, _p(s), s_stride_row,
                                   s_stride_group, _p(h_out), ld_h, _stream(stream))
    return _check("fp8_silu_mul_quant", st, raise_on_error)


def fp8_moe_combine(y, rows, H, ld_y, token_rows, weights, T, k, out, ld_out, out_type, stream=None,
                    raise_on_error=True):
    st = load().fp8_moe_combine(_p(y), rows, H, ld_y, _p(token_rows), _p(weights), T, k, _p(out), ld_out,
                                out_type, _stream(stream))
    return _check("fp8_moe_combine", st, raise_on_error)


def fp8_moe_combine_routed(y, rows, H, ld_y, token_rows, weights, T, k, out, ld_out, out_type, stream=None,
                           raise_on_error=True):
    st = load().fp8_moe_combine_routed(_p(y), rows, H, ld_y, _p(token_rows), _p(weights), T, k, _p(out), ld_out,
                                       out_type, _stream(stream))
    return _check("fp8_moe_combine_routed", st, raise_on_error)


def fp8_moe_combine_backward(dout, ld_dout, dout_type, y, rows, H, ld_y, token_rows, weights, T, k, dy, ld_dy,
                             dweights, stream=None, raise_on_error=True):
    st = load().fp8_moe_combine_backward(_p(dout), ld_dout, dout_type, _p(y), rows, H, ld_y, _p(token_rows),
                                         _p(weights), T, k, _p(dy), ld_dy, _p(dweights), _stream(stream))
    return _check("fp8_moe_combine_backward", st, raise_on_error)


def fp8_moe_route(logits, T, E, ld, type_, k, renorm, mask, experts, weights, counts, offsets, row_token, token_rows,
                  lse, loss, ws, ws_bytes, stream=None, raise_on_error=True):
    st = load().fp8_moe_route(_p(logits), T, E, ld, type_, k, renorm, _p(mask), _p(experts), _p(weights), _p(counts),
                              _p(offsets), _p(row_token), _p(token_rows), _p(lse), _p(loss), _p(ws), ws_bytes,
                              _stream(stream))
    return _check("fp8_moe_route", st, raise_on_error)


def fp8_moe_route_ws_size(T, E):
    """Workspace bytes of fp8_moe_route (host only)."""
    out = ctypes.c_size_t(0)
    _check("fp8_moe_route_ws_size", load().fp8_moe_route_ws_size(T, E, ctypes.byref(out)))
    return out.value


def fp8_moe_route_backward(logits, T, E, ld, type_, k, renorm, experts, weights, counts, lse, dweights, dloss,
                           dlogits, ld_d, stream=None, raise_on_error=True):
    st = load().fp8_moe_route_backward(_p(logits), T, E, ld, type_, k, renorm, _p(experts), _p(weights), _p(counts),
                                       _p(lse), _p(dweights), _p(dloss), _p(dlogits), ld_d, _stream(stream))
    return _check("fp8_moe_route_backward", st, raise_on_error)


def fp8_moe_route_grouped(logits, T, E, ld, type_, k, score, bias, groups, keep_groups, group_score, renorm, scale, mask,
                          experts, weights, counts, offsets, row_token, token_rows, total, loss, ws, ws_bytes,
                          stream=None, raise_on_error=True):
    st = load().fp8_moe_route_grouped(_p(logits), T, E, ld, type_, k, score, _p(bias), groups, keep_groups, group_score,
                                      renorm, scale, _p(mask), _p(experts), _p(weights), _p(counts), _p(offsets),
                                      _p(row_token), _p(token_rows), _p(total), _p(loss), _p(ws), ws_bytes,
                                      _stream(stream))
    return _check("fp8_moe_route_grouped", st, raise_on_error)


def fp8_moe_route_grouped_backward(logits, T, E, ld, type_, k, score, renorm, scale, experts, counts, total, dweights,
                                   dloss, dlogits, ld_d, stream=None, raise_on_error=True):
    st = load().fp8_moe_route_grouped_backward(_p(logits), T, E, ld, type_, k, score, renorm, scale, _p(experts),
                                               _p(counts), _p(total), _p(dweights), _p(dloss), _p(dlogits), ld_d,
                                               _stream(stream))
    return _check("fp8_moe_route_grouped_backward", st, raise_on_error)


def fp8_moe_bias_update(bias, counts, E, rate, stream=None, raise_on_error=True):
    st = load().fp8_moe_bias_update(_p(bias), _p(counts), E, rate, _stream(stream))
    return _check("fp8_moe_bias_update", st, raise_on_error)


def fp8_block_norm(rows, cols, x, ld_x, residual, ld_r, stream_type, gate, ld_gate, rows_per_gate, scale, w_post,
                   w_pre, w_type, eps, h, ld_h, y, ld_y, q, ld_q, s, s_stride_row, s_stride_group, stream=None,
                   raise_on_error=True):
    st = load().fp8_block_norm(rows, cols, _p(x), ld_x, _p(residual), ld_r, stream_type, _p(gate), ld_gate,
                               rows_per_gate, scale, _p(w_post), _p(w_pre), w_type, eps, _p(h), ld_h, _p(y), ld_y,
                               _p(q), ld_q, _p(s), s_stride_row, s_stride_group, _stream(stream))
    return _check("fp8_block_norm", st, raise_on_error)


def fp8_block_norm_backward(rows, cols, dy, ld_dy, dy_type, dh, ld_dh, h, ld_h, stream_type, x, ld_x, gate, ld_gate,
                            rows_per_gate, scale, w_post, w_pre, w_type, eps, dx, ld_dx, dres, ld_dres, dgate,
                            ld_dgate, dgate_type, dw_post, dw_pre, ws, ws_bytes, stream=None, raise_on_error=True):
    st = load().fp8_block_norm_backward(rows, cols, _p(dy), ld_dy, dy_type, _p(dh), ld_dh, _p(h), ld_h, stream_type,
                                        _p(x), ld_x, _p(gate), ld_gate, rows_per_gate, scale, _p(w_post), _p(w_pre),
                                        w_type, eps, _p(dx), ld_dx, _p(dres), ld_dres, _p(dgate), ld_dgate,
                                        dgate_type, _p(dw_post), _p(dw_pre), _p(ws), ws_bytes, _stream(stream))
    return _check("fp8_block_norm_backward", st, raise_on_error)


def fp8_block_norm_backward_ws_size(rows, cols, rows_per_gate, dw_post, dw_pre, dgate):
    """Workspace bytes of fp8_block_norm_backward (host only)."""
    out = ctypes.c_size_t(0)
    _check("fp8_block_norm_backward_ws_size",
           load().fp8_block_norm_backward_ws_size(rows, cols, rows_per_gate, int(dw_post), int(dw_pre), int(dgate),
                                                  ctypes.byref(out)))
    return out.value


def mxfp8_quant(x, rows, cols, ld_x, q, ld_q, s, s_stride_row, s_stride_group, stream=None, raise_on_error=True):
    st = load().mxfp8_quant(_p(x), rows, cols, ld_x, _p(q), ld_q, _p(s), s_stride_row, s_stride_group,
                            _stream(stream))
    return _check("mxfp8_quant", st, raise_on_error)


def mxfp8_quant_t(x, rows, cols, ld_x, qt, ld_qt, s, s_stride_row, s_stride_group, stream=None,
                  raise_on_error=True):
    st = load().mxfp8_quant_t(_p(x), rows, cols, ld_x, _p(qt), ld_qt, _p(s), s_stride_row, s_stride_group,
                              _stream(stream))
    return _check("mxfp8_quant_t", st, raise_on_error)


def fp8_quant_dual_axis(x, rows, cols, ld_x, mx, q, ld_q, s, s_stride_row, s_stride_group, qt, ld_qt, st,
                        st_stride_row, st_stride_group, stream=None, raise_on_error=True):
    r = load().fp8_quant_dual_axis(_p(x), rows, cols, ld_x, mx, _p(q), ld_q, _p(s), s_stride_row, s_stride_group,
                                   _p(qt), ld_qt, _p(st), st_stride_row, st_stride_group, _stream(stream))
    return _check("fp8_quant_dual_axis", r, raise_on_error)


def fp8_quant_linear_pow2(x, rows, cols, ld_x, qx, ld_qx, sx, ld_sx, w, w_rows, ld_w, qw, ld_qw, sw, ld_sw,
                          stream=None, raise_on_error=True):
    r = load().fp8_quant_linear_pow2(_p(x), rows, cols, ld_x, _p(qx), ld_qx, _p(sx), ld_sx, _p(w), w_rows, ld_w,
                                     _p(qw), ld_qw, _p(sw), ld_sw, _stream(stream))
    return _check("fp8_quant_linear_pow2", r, raise_on_error)


def fp8_transpose_codes(q, batch, rows, cols, ld_q, q_t, ld_qt, stream=None, raise_on_error=True):
    r = load().fp8_transpose_codes(_p(q), batch, rows, cols, ld_q, _p(q_t), ld_qt, _stream(stream))
    return _check("fp8_transpose_codes", r, raise_on_error)


def fp8_quant_pow2(x, rows, cols, ld_x, block_rows, q, ld_q, s, ld_s, stream=None, raise_on_error=True):
    st = load().fp8_quant_pow2(_p(x), rows, cols, ld_x, block_rows, _p(q), ld_q, _p(s), ld_s, _stream(stream))
    return _check("fp8_quant_pow2", st, raise_on_error)


def fp8_blockscaled_gemm_pow2(M, N, K, a, lda, sa, lds_a, b, ldb, sb, lds_b, c, ldc, out, stream=None,
                              raise_on_error=True):
    st = load().fp8_blockscaled_gemm_pow2(M, N, K, _p(a), lda, _p(sa), lds_a, _p(b), ldb, _p(sb), lds_b, _p(c), ldc,
                                          out, _stream(stream))
    return _check("fp8_blockscaled_gemm_pow2", st, raise_on_error)


def mxfp8_gemm(rows, N, K, G, offsets, a_rows, a_count, a, lda, sa, lds_a, b, ldb, b_stride_g, sb, lds_b,
               sb_stride_g, c, ldc, out, stream=None, raise_on_error=True):
    st = load().mxfp8_gemm(rows, N, K, G, _p(offsets), _p(a_rows), a_count, _p(a), lda, _p(sa), lds_a, _p(b), ldb,
                           b_stride_g, _p(sb), lds_b, sb_stride_g, _p(c), ldc, out, _stream(stream))
    return _check("mxfp8_gemm", st, raise_on_error)


def int8_quant(x, rows, cols, ld_x, axis, q, ld_q, s, stream=None, raise_on_error=True):
    st = load().int8_quant(_p(x), rows, cols, ld_x, axis, _p(q), ld_q, _p(s), _stream(stream))
    return _check("int8_quant", st, raise_on_error)


def int8_silu_mul_quant(gate_up, rows, I, ld_in, live_rows, q, ld_q, s, h_out, ld_h, stream=None,
                        raise_on_error=True):
    st = load().int8_silu_mul_quant(_p(gate_up), rows, I, ld_in, _p(live_rows), _p(q), ld_q, _p(s), _p(h_out), ld_h,
                                    _stream(stream))
    return _check("int8_silu_mul_quant", st, raise_on_error)


def int8_gemm(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, out, ws, ws_bytes, stream=None, raise_on_error=True):
    st = load().int8_gemm(M, N, K, _p(a), lda, _p(sa), _p(b), ldb, _p(sb), _p(c), ldc, out, _p(ws), ws_bytes,
                          _stream(stream))
    return _check("int8_gemm", st, raise_on_error)


def int8_gemm_ws_size(M, N, K):
    """Workspace bytes that int8_gemm has use for (host only)."""
    out = ctypes.c_size_t(0)
    _check("int8_gemm_ws_size", load().int8_gemm_ws_size(M, N, K, ctypes.byref(out)))
    return out.value


def int8_linear(rows, N, cols, x, ld_x, w, ld_w, sw, y, ld_y, out, ws, ws_bytes, stream=None, raise_on_error=True):
    st = load().int8_linear(rows, N, cols, _p(x), ld_x, _p(w), ld_w, _p(sw), _p(y), ld_y, out, _p(ws), ws_bytes,
                            _stream(stream))
    return _check("int8_linear", st, raise_on_error)


def int8_linear_ws_size(rows, N, cols):
    """Workspace bytes of int8_linear (host only)."""
    out = ctypes.c_size_t(0)
    _check("int8_linear_ws_size", load().int8_linear_ws_size(rows, N, cols, ctypes.byref(out)))
    return out.value


def int8_linear_backward(T, O, I, dy, ld_dy, w, ld_w, x, ld_x, dx, ld_dx, dw, ld_dw, ws, ws_bytes, stream=None,
                         raise_on_error=True):
    st = load().int8_linear_backward(T, O, I, _p(dy), ld_dy, _p(w), ld_w, _p(x), ld_x, _p(dx), ld_dx, _p(dw), ld_dw,
                                     _p(ws), ws_bytes, _stream(stream))
    return _check("int8_linear_backward", st, raise_on_error)


def int8_linear_backward_ws_size(T, O, I):
    """Workspace bytes of int8_linear_backward (host only)."""
    out = ctypes.c_size_t(0)
    _check("int8_linear_backward_ws_size", load().int8_linear_backward_ws_size(T, O, I, ctypes.byref(out)))
    return out.value


def int8_grouped_gemm(total_rows, N, K, G, offsets, a_rows, a_count, a, lda, sa, b, ldb, b_stride_g, sb, sb_stride_g,
                      c, ldc, out, stream=None, raise_on_error=True):
    st = load().int8_grouped_gemm(total_rows, N, K, G, _p(offsets), _p(a_rows), a_count, _p(a), lda, _p(sa), _p(b),
                                  ldb, b_stride_g, _p(sb), sb_stride_g, _p(c), ldc, out, _stream(stream))
    return _check("int8_grouped_gemm", st, raise_on_error)


def fp8bs_e4m3_encode(inp, out, n, stream=None, raise_on_error=True):
    st = load().fp8bs_e4m3_encode(_p(inp), _p(out), n, _stream(stream))
    return _check("fp8bs_e4m3_encode", st, raise_on_error)


# ------------------------------------------------------- tensor conveniences
def _u8(shape, device):
    return torch.empty(shape, dtype=torch.uint8, device=device)


def quant_rowblock(x: torch.Tensor, axis: int = AXIS_ROW, scale_layout: str = "m_major"):
    """Quantize a bf16 [rows, cols] tensor.  Returns (q, s) with s logically
    [rows, groups] (AXIS_ROW) or [cols, groups] (AXIS_COL).  scale_layout
    'm_major' stores s as a [groups, rows] buffer (stride_row 1) and returns a
    [rows, groups] view of it; 'row_major' stores [rows, groups]."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if axis == AXIS_ROW:
        q = _u8((rows, cols), x.device)
        lead, ng = rows, (cols + 127) // 128
        ld_q = cols
    else:
        q = _u8((cols, rows), x.device)
        lead, ng = cols, (rows + 127) // 128
        ld_q = rows
    if scale_layout == "m_major":
        sbuf = torch.empty((ng, lead), dtype=torch.float32, device=x.device)
        s, ssr, ssg = sbuf.t(), 1, lead
    else:
        s = torch.empty((lead, ng), dtype=torch.float32, device=x.device)
        ssr, ssg = ng, 1
    fp8_quant_rowblock(x, rows, cols, x.stride(0), axis, q, ld_q, s, ssr, ssg)
    return q, s


def quant_dual_axis(x: torch.Tensor, mx: bool = False):
    """Row groups and column groups of a bf16 [rows, cols] tensor from one
    read: (q [rows, cols], s, qt [cols, rows], st).  FP32 scales (mx False):
    s is a [rows, cols/128] view of a [cols/128, rows] buffer and st a
    [cols, rows/128] view of a [rows/128, cols] buffer (the M-major layouts
    the GEMMs read); MX: uint8 s [rows, cols/32] and st [cols, rows/32],
    row-major."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    q, qt = _u8((rows, cols), x.device), _u8((cols, rows), x.device)
    if mx:
        s, st = _u8((rows, cols // 32), x.device), _u8((cols, rows // 32), x.device)
        fp8_quant_dual_axis(x, rows, cols, x.stride(0), 1, q, cols, s, cols // 32, 1, qt, rows, st, rows // 32, 1)
        return q, s, qt, st
    ng, ngt = (cols + 127) // 128, (rows + 127) // 128
    sbuf = torch.empty((ng, rows), dtype=torch.float32, device=x.device)
    stbuf = torch.empty((ngt, cols), dtype=torch.float32, device=x.device)
    fp8_quant_dual_axis(x, rows, cols, x.stride(0), 0, q, cols, sbuf, 1, rows, qt, rows, stbuf, 1, cols)
    return q, sbuf.t(), qt, stbuf.t()


def quant_linear(x: torch.Tensor, w: torch.Tensor):
    """Both operands of a linear layer in one launch: X [rows, cols] in 1x128
    groups (M-major scales, returned as a [rows, groups] view) and W
    [w_rows, cols] in 128x128 blocks.  Returns (qx, sx, qw, sw)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_contiguous()
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.is_contiguous() and w.shape[1] == x.shape[1]
    rows, cols = x.shape
    w_rows = w.shape[0]
    ng = (cols + 127) // 128
    qx, qw = _u8((rows, cols), x.device), _u8((w_rows, cols), x.device)
    sbuf = torch.empty((ng, rows), dtype=torch.float32, device=x.device)
    sw = torch.empty(((w_rows + 127) // 128, ng), dtype=torch.float32, device=x.device)
    fp8_quant_linear(x, rows, cols, cols, qx, cols, sbuf, 1, rows, w, w_rows, cols, qw, cols, sw)
    return qx, sbuf.t(), qw, sw


def quant_block2d(w: torch.Tensor, transposed: bool = False):
    """128x128 block quantization of a bf16 [rows, cols] or [batch, rows, cols]
    tensor.  Returns (q, s, q_t or None)."""
    assert w.dtype == torch.bfloat16 and w.is_contiguous()
    batched = w.dim() == 3
    ww = w if batched else w.unsqueeze(0)
    batch, rows, cols = ww.shape
    q = _u8(ww.shape, w.device)
    qt = _u8((batch, cols, rows), w.device) if transposed else None
    s = torch.empty((batch, (rows + 127) // 128, (cols + 127) // 128), dtype=torch.float32, device=w.device)
    fp8_quant_block2d(ww, batch, rows, cols, cols, q, cols, qt, rows, s)
    if not batched:
        q, s = q[0], s[0]
        qt = qt[0] if qt is not None else None
    return q, s, qt


def quant_rowwise(x: torch.Tensor):
    """One scale per row of a bf16 [rows, cols] tensor -> (q, s [rows])."""
    rows, cols = x.shape
    q = _u8((rows, cols), x.device)
    s = torch.empty((rows,), dtype=torch.float32, device=x.device)
    fp8_quant_rowwise(x, rows, cols, x.stride(0), q, cols, s)
    return q, s


def quant_tensorwise(x: torch.Tensor):
    """One scale for a whole bf16 [rows, cols] tensor -> (q, s [1])."""
    rows, cols = x.shape
    q = _u8((rows, cols), x.device)
    s = torch.empty((1,), dtype=torch.float32, device=x.device)
    fp8_quant_tensorwise(x, rows, cols, x.stride(0), q, cols, s)
    return q, s


def gemm_rowscaled(a, sa, b, sb, out_dtype=torch.bfloat16):
    """C = diag(sa) (A B^T) diag(sb) for codes a [M, K], b [N, K] and scales
    sa [M] or [1], sb [N] or [1] (rowwise or tensorwise): the block-scaled GEMM
    with scale views of K stride 0."""
    M, K = a.shape
    N = b.shape[0]
    sa_v = sa.view(-1, 1).expand(M, K // 128)
    sb_v = sb.view(-1, 1).expand(N, K // 128)
    return gemm(a, sa_v, b, sb_v, bscale=BSCALE_ROW128, out_dtype=out_dtype)


def gemm(a, sa, b, sb, bscale=BSCALE_BLOCK128, out_dtype=torch.bfloat16):
    """C = A B^T for codes a [M, K], b [N, K] and logical scale views
    sa [M, K/128], sb [N/128 or N, K/128] (any strides)."""
    M, K = a.shape
    N = b.shape[0]
    c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    fp8_blockscaled_gemm(M, N, K, a, a.stride(0), sa, sa.stride(0), sa.stride(1), b, b.stride(0), sb, sb.stride(0),
                         sb.stride(1), bscale, c, c.stride(0), OUT_FP32 if out_dtype == torch.float32 else OUT_BF16)
    return c


def linear_forward(x: torch.Tensor, w: torch.Tensor, out_dtype=torch.bfloat16):
    """Y = X W^T of the block-wise FP8 linear layer: X [T, in] in 1x128 groups
    and W [out, in] in 128x128 blocks (one launch), then the block-scaled GEMM.
    Returns (y, saved); saved = (qw, sw, x) is what linear_backward reads: the
    weight's codes and scales (dgrad's operand is their transpose) and the
    bf16 activation (quantized along tokens for wgrad)."""
    qx, sx, qw, sw = quant_linear(x, w)
    return gemm(qx, sx, qw, sw, BSCALE_BLOCK128, out_dtype), (qw, sw, x)


def linear_backward(dy: torch.Tensor, saved):
    """dX = dY W and dW = dY^T X, both fp32, of the layer linear_forward ran:
    dY [T, out] in 1x128 groups (dgrad) and 128x1 groups along tokens (wgrad)
    from one read, X in 128x1 groups along tokens, and W^T as the transposed
    copy of the forward's codes with W's 128x128 scales read transposed."""
    qw, sw, x = saved
    assert dy.dtype == torch.bfloat16 and dy.dim() == 2 and dy.is_contiguous()
    T, O = dy.shape
    I = x.shape[1]
    qdy, sdy, qdyt, sdyt = quant_dual_axis(dy)
    qxt, sxt = quant_rowblock(x, AXIS_COL, "m_major")
    qwt = _u8((I, O), dy.device)
    fp8_transpose_codes(qw, 1, O, I, qw.stride(0), qwt, O)
    dx = gemm(qdy, sdy, qwt, sw.t(), BSCALE_BLOCK128, torch.float32)
    dw = gemm(qdyt, sdyt, qxt, sxt, BSCALE_ROW128, torch.float32)
    return dx, dw


def _moe_experts(qx, sx, T, qgu, sgu, qdt, sdt, offsets, row_token):
    """The experts' MLPs over the routed rows of a quantized activation: y
    bf16 [rows, H] in expert-sorted order."""
    G, N2, H = qgu.shape
    I = N2 // 2
    rows = row_token.numel()
    dev = qx.device
    # the products walk the experts by these sizes: anything else would be read past its end
    for name, t, shape in (("qgu", qgu, (G, 2 * I, qx.shape[1])), ("qdt", qdt, (G, H, I))):
        if t.shape != shape or t.element_size() != 1 or not t.is_contiguous() or t.device != dev:
            raise ValueError("%s: contiguous codes %s on %s expected, got %s %s, strides %s, on %s"
                             % (name, list(shape), dev, t.dtype, tuple(t.shape), t.stride(), t.device))
    ng = lambda n: (n + 127) // 128
    for name, t, shape in (("sgu", sgu, (G, ng(N2), ng(H))), ("sdt", sdt, (G, ng(I), ng(H)))):
        if t.shape != shape or t.dtype is not torch.float32 or t.device != dev:
            raise ValueError("%s: float32 %s on %s expected, got %s %s on %s"
                             % (name, list(shape), dev, t.dtype, tuple(t.shape), t.device))
    qh = _u8((rows, I), dev)
    shb = torch.empty((I // 128, rows), dtype=torch.float32, device=dev)
    fp8_grouped_gemm_swiglu_quant(rows, I, H, G, offsets, row_token, T, qx, qx.stride(0) if T > 1 else H, sx,
                                  sx.stride(0), sx.stride(1), qgu, H, N2 * H, sgu, sgu.stride(0), sgu.stride(1),
                                  sgu.stride(2), qh, I, shb, 1, rows)
    y = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
    fp8_grouped_gemm(rows, H, I, G, offsets, None, rows, qh, I, shb, 1, rows, qdt, I, H * I, sdt, sdt.stride(0),
                     sdt.stride(2), sdt.stride(1), y, H, OUT_BF16)
    return y


def moe_forward(x, qgu, sgu, qdt, sdt, offsets, row_token, token_rows, weights, out_dtype=torch.bfloat16):
    """One block-wise FP8 MoE layer forward: X [T, H] in 1x128 groups; the
    grouped gate/up GEMM over the experts' rows (gathered by row_token), with
    SiLU*mul and the 1x128 requantization of h in its epilogue; the grouped
    down GEMM; the routing-weighted combine.  Weights come quantized:
    qgu [G, 2I, H] codes with sgu [G, 2I/128, H/128] (gate rows [0, I), up
    rows [I, 2I)), qdt [G, H, I] codes of the down weights ([out][in]) with
    sdt [G, I/128, H/128] (the blocks of the [in][out] stack, read transposed).
    offsets int32 [G + 1] (device), row_token int32 [rows], token_rows int32
    [T, k] (grouped row of each token's slot), weights fp32 [T, k]."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_contiguous()
    T, H = x.shape
    rows = row_token.numel()
    qx, sx = quant_rowblock(x, AXIS_ROW, "m_major")
    y = _moe_experts(qx, sx, T, qgu, sgu, qdt, sdt, offsets, row_token)
    k = token_rows.shape[1]
    out = torch.empty((T, H), dtype=out_dtype, device=x.device)
    fp8_moe_combine(y, rows, H, H, token_rows.contiguous(), weights.contiguous(), T, k, out, H,
                    OUT_FP32 if out_dtype == torch.float32 else OUT_BF16)
    return out


def moe_forward_routed(codes, logits, top_k, qgu, sgu, qdt, sdt, *, renorm=True, mask=None,
                       out_dtype=torch.bfloat16, router: Optional[dict] = None):
    """One block-wise FP8 MoE layer from router logits [T, G]: moe_route (or, with
    `router`, moe_route_grouped with those options), the experts on the
    activation's codes, the combine.  codes = (q [T, H] with
    unit column stride, s [T, H/128]) as quant_rowblock or block_norm give
    them; weights as in moe_forward.  Masked tokens reach no expert and get zeros.  Returns (out
    [T, H], routing, y): y is the experts' output, which
    moe_combine_backward reads."""
    qx, sx = codes
    T, H = qx.shape
    G, N2, Hw = qgu.shape
    if logits.shape != (T, G):
        raise ValueError("logits: [%d, %d] expected, got %s" % (T, G, tuple(logits.shape)))
    if H != Hw or qdt.shape != (G, H, N2 // 2):
        raise ValueError("codes of %d columns, experts of %s and %s" % (H, tuple(qgu.shape), tuple(qdt.shape)))
    _mat("codes", qx, T, H, _device(), torch.uint8)
    if sx.dtype is not _F32 or sx.shape != (T, (H + 127) // 128) or sx.get_device() != _device():
        raise ValueError("scales of the codes: float32 [%d, %d] on cuda:%d expected, got %s %s on %s"
                         % (T, (H + 127) // 128, _device(), sx.dtype, tuple(sx.shape), sx.device))
    if router is None:
        r = moe_route(logits, top_k, renorm=renorm, mask=mask)
    else:
        r = moe_route_grouped(logits, top_k, renorm=renorm, mask=mask, **router)
    y = _moe_experts(qx, sx, T, qgu, sgu, qdt, sdt, r.offsets, r.row_token)
    out = torch.empty((T, H), dtype=out_dtype, device=qx.device)
    fp8_moe_combine_routed(y, T * top_k, H, H, r.token_rows, r.weights, T, top_k, out, H, _otype(out_dtype))
    return out, r, y


# ---------------------------------- between the GEMMs: norms and the router
# The smallest of these kernels run for 4 to 6 us and a launch costs 3, so the
# conveniences below keep their own part short: one check per tensor, pointers
# passed as plain integers.
_BF, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_OTYPES = {_BF: OUT_BF16, _F32: OUT_FP32}


def _otype(dtype):
    t = _OTYPES.get(dtype)
    if t is None:
        raise TypeError("bfloat16 or float32 expected, got %s" % dtype)
    return t


def _device():
    return torch.cuda.current_device()


def _mat(name, t, rows, cols, dev, dt, dt2=None):
    """(pointer, leading dimension) of a [rows, cols] tensor of type dt or dt2
    with unit column stride on the current device; (None, 0) without one."""
    if t is None:
        return None, 0
    d = t.dtype
    if (d is dt or d is dt2) and t.shape == (rows, cols) and t.get_device() == dev:
        s0, s1 = t.stride()
        if s1 == 1 or cols <= 1:
            return t.data_ptr(), s0 if rows > 1 else cols      # the stride of a single row is never used
    raise ValueError("%s: [%d, %d] of %s with unit column stride on cuda:%d expected, got %s %s, strides %s, on %s"
                     % (name, rows, cols, dt if dt2 is None else "%s or %s" % (dt, dt2), dev, tuple(t.shape), d,
                        t.stride(), t.device))


def _arr(name, t, shape, dev, dt):
    """Pointer of a contiguous tensor of this shape and type on the current
    device; None without one."""
    if t is None:
        return None
    if t.dtype is dt and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s: contiguous %s %s on cuda:%d expected, got %s %s on %s"
                     % (name, dt, list(shape), dev, t.dtype, tuple(t.shape), t.device))


def _workspace(ws, dev):
    """(pointer, bytes) of a workspace; the call itself checks its size."""
    if ws is None:
        return None, 0
    return _arr("ws", ws, ws.shape, dev, torch.uint8), ws.numel()


class BlockNorm(NamedTuple):
    """Outputs of block_norm (None where not asked for).  s is a [rows,
    groups] view of a [groups, rows] buffer, the layout the GEMMs read."""
    h: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    s: Optional[torch.Tensor]


def block_norm(residual=None, x=None, *, w_pre=None, w_post=None, gate=None, rows_per_gate=1, scale=1.0, eps=1e-6,
               h=True, y=True, quant=True, out: Optional[BlockNorm] = None) -> BlockNorm:
    """h = residual + scale * gate * N(x; w_post) and y = N(h; w_pre) with
    1x128 E4M3 codes (q, s) for the next linear layer, in one pass (see
    fp8_block_norm).  residual [rows, cols] bf16 or fp32 and x bf16 (one of
    them may be missing), gate bf16 [ceil(rows / rows_per_gate), cols], weights
    bf16 or fp32 [cols].  h, y, quant say which outputs to make (y and quant
    only with w_pre; h takes the residual's type); `out` is an earlier result
    of the same call whose tensors are written again."""
    ref = x if residual is None else residual
    if ref is None:
        raise ValueError("residual or x is required")
    rows, cols = ref.shape
    dev, ng = _device(), (cols + 127) // 128
    stream_dt = _BF if residual is None else residual.dtype
    stype = _otype(stream_dt)
    rp, ld_r = _mat("residual", residual, rows, cols, dev, stream_dt)
    xp, ld_x = _mat("x", x, rows, cols, dev, _BF)
    gp = ld_g = None
    if gate is not None:
        if rows_per_gate < 1:
            raise ValueError("rows_per_gate must be >= 1")
        gp, ld_g = _mat("gate", gate, -(-rows // rows_per_gate), cols, dev, _BF)
    w = w_post if w_pre is None else w_pre
    wdt = _BF if w is None else w.dtype
    pre, post = _arr("w_pre", w_pre, (cols,), dev, wdt), _arr("w_post", w_post, (cols,), dev, wdt)
    if w_pre is None:
        y = quant = False
    if out is None:
        e = lambda *shape, dt: torch.empty(shape, dtype=dt, device=ref.device)
        out = BlockNorm(e(rows, cols, dt=stream_dt) if h else None, e(rows, cols, dt=_BF) if y else None,
                        e(rows, cols, dt=torch.uint8) if quant else None, e(ng, rows, dt=_F32).t() if quant else None)
    ho, yo, qo, so = out
    if (ho is None) is bool(h) or (yo is None) is bool(y) or (qo is None) is bool(quant):
        raise ValueError("out does not hold the outputs asked for")
    hp, ld_h = _mat("out.h", ho, rows, cols, dev, stream_dt)
    yp, ld_y = _mat("out.y", yo, rows, cols, dev, _BF)
    qp, ld_q = _mat("out.q", qo, rows, cols, dev, torch.uint8)
    sp = ssr = ssg = 0
    if qo is not None:
        if so is None or so.dtype is not _F32 or so.shape != (rows, ng) or so.get_device() != dev:
            raise ValueError("out.s: float32 [%d, %d] on cuda:%d expected" % (rows, ng, dev))
        sp, (ssr, ssg) = so.data_ptr(), so.stride()
    st = load().fp8_block_norm(rows, cols, xp, ld_x, rp, ld_r, stype, gp, ld_g or 0, rows_per_gate, scale, post, pre,
                               _otype(wdt), eps, hp, ld_h, yp, ld_y, qp, ld_q, sp or None, ssr, ssg, _stream())
    if st:
        _check("fp8_block_norm", st)
    return out


class BlockNormGrads(NamedTuple):
    """Outputs of block_norm_backward (None where there is nothing to give);
    ws is the call's workspace."""
    dres: Optional[torch.Tensor]
    dx: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]
    ws: Optional[torch.Tensor]


def block_norm_backward(dy=None, dh=None, h=None, x=None, *, w_pre=None, w_post=None, gate=None, rows_per_gate=1,
                        scale=1.0, eps=1e-6, dres=True, dgate_dtype=torch.float32,
                        out: Optional[BlockNormGrads] = None) -> BlockNormGrads:
    """Gradients of block_norm from dy = dL/dy (bf16 or fp32; with h and
    w_pre) and dh = dL/dh past y (h's type), at the saved h and x: dres (the
    stream's type; not made with dres=False), dx bf16 when there is an x, dgate
    (dgate_dtype) when there is a gate, dw_post and dw_pre fp32.  `out` is an
    earlier result of the same call whose tensors are written again."""
    ref = dh if dh is not None else h
    if ref is None:
        raise ValueError("dh, or dy with h, is required")
    rows, cols = ref.shape
    dev = _device()
    stream_dt = ref.dtype
    stype = _otype(stream_dt)
    if (dy is None) is not (w_pre is None) or (dy is None) is not (h is None):
        raise ValueError("dy, h and w_pre go together")
    if x is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate need x")
    dyp, ld_dy = _mat("dy", dy, rows, cols, dev, _BF, _F32)
    dhp, ld_dh = _mat("dh", dh, rows, cols, dev, stream_dt)
    hp, ld_h = _mat("h", h, rows, cols, dev, stream_dt)
    xp, ld_x = _mat("x", x, rows, cols, dev, _BF)
    gp, ld_g, ngate = None, 0, 0
    if gate is not None:
        if rows_per_gate < 1:
            raise ValueError("rows_per_gate must be >= 1")
        ngate = -(-rows // rows_per_gate)
        gp, ld_g = _mat("gate", gate, ngate, cols, dev, _BF)
    w = w_post if w_pre is None else w_pre
    wdt = _BF if w is None else w.dtype
    pre, post = _arr("w_pre", w_pre, (cols,), dev, wdt), _arr("w_post", w_post, (cols,), dev, wdt)
    if out is None:
        need = fp8_block_norm_backward_ws_size(rows, cols, rows_per_gate, w_post is not None, w_pre is not None,
                                               gate is not None)
        e = lambda *shape, dt: torch.empty(shape, dtype=dt, device=ref.device)
        out = BlockNormGrads(e(rows, cols, dt=stream_dt) if dres else None,
                             None if x is None else e(rows, cols, dt=_BF),
                             None if gate is None else e(ngate, cols, dt=dgate_dtype),
                             None if w_post is None else e(cols, dt=_F32), None if w_pre is None else e(cols, dt=_F32),
                             e(need, dt=torch.uint8) if need else None)
    o_dres, o_dx, o_dgate, o_post, o_pre, ws = out
    if ((o_dres is None) is bool(dres) or (o_dx is None) is not (x is None) or (o_dgate is None) is not (gate is None)
            or (o_post is None) is not (w_post is None) or (o_pre is None) is not (w_pre is None)):
        raise ValueError("out does not hold the outputs of this call")
    drp, ld_dres = _mat("out.dres", o_dres, rows, cols, dev, stream_dt)
    dxp, ld_dx = _mat("out.dx", o_dx, rows, cols, dev, _BF)
    dgp, ld_dg = _mat("out.dgate", o_dgate, ngate, cols, dev, dgate_dtype)
    dpost, dpre = _arr("out.dw_post", o_post, (cols,), dev, _F32), _arr("out.dw_pre", o_pre, (cols,), dev, _F32)
    wsp, wsn = _workspace(ws, dev)
    st = load().fp8_block_norm_backward(rows, cols, dyp, ld_dy, OUT_FP32 if dy is not None and dy.dtype is _F32 else
                                        OUT_BF16, dhp, ld_dh, hp, ld_h, stype, xp, ld_x, gp, ld_g, rows_per_gate,
                                        scale, post, pre, _otype(wdt), eps, dxp, ld_dx, drp, ld_dres, dgp, ld_dg,
                                        _otype(dgate_dtype), dpost, dpre, wsp, wsn, _stream())
    if st:
        _check("fp8_block_norm_backward", st)
    return out


class Routing(NamedTuple):
    """Outputs of moe_route: int32 experts [T, k] (-1: none), fp32 weights
    [T, k], int32 counts [E + 1] (the last one: routed tokens), offsets
    [E + 1], row_token [T * k], token_rows [T, k] (-1: no row), fp32 lse [T]
    and loss [2] (balance, z); ws is the call's workspace."""
    experts: torch.Tensor
    weights: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    row_token: torch.Tensor
    token_rows: torch.Tensor
    lse: torch.Tensor
    loss: torch.Tensor
    ws: Optional[torch.Tensor]


def _routing(logits, T, E, tk, dev, out):
    """(Routing, pointers of its tensors in the entry points' order, workspace and
    its size behind them)."""
    if out is None:
        need = fp8_moe_route_ws_size(T, E)
        e = lambda *shape, dt=_I32: torch.empty(shape, dtype=dt, device=logits.device)
        out = Routing(e(*tk), e(*tk, dt=_F32), e(E + 1), e(E + 1), e(T * tk[1]), e(*tk), e(T, dt=_F32), e(2, dt=_F32),
                      e(need, dt=torch.uint8) if need else None)
    experts, weights, counts, offsets, row_token, token_rows, lse, loss, ws = out
    return out, (_arr("out.experts", experts, tk, dev, _I32), _arr("out.weights", weights, tk, dev, _F32),
                 _arr("out.counts", counts, (E + 1,), dev, _I32), _arr("out.offsets", offsets, (E + 1,), dev, _I32),
                 _arr("out.row_token", row_token, (T * tk[1],), dev, _I32),
                 _arr("out.token_rows", token_rows, tk, dev, _I32), _arr("out.lse", lse, (T,), dev, _F32),
                 _arr("out.loss", loss, (2,), dev, _F32), *_workspace(ws, dev))


def moe_route(logits, top_k, *, renorm=True, mask=None, out: Optional[Routing] = None) -> Routing:
    """Top-k routing of router logits [T, E] (bf16 or fp32): experts, weights,
    counts, the expert-sorted row maps of moe_forward and the grouped GEMMs,
    and the balance and z losses (see fp8_moe_route).  mask [T] (bool or
    uint8): tokens with False are not routed.  `out` is an earlier result for
    the same sizes whose tensors are written again."""
    T, E = logits.shape
    dev, tk = _device(), (T, top_k)
    zp, ld = _mat("logits", logits, T, E, dev, _BF, _F32)
    mp = None if mask is None else _arr("mask", mask, (T,), dev, mask.dtype if mask.dtype is torch.bool else torch.uint8)
    out, ptrs = _routing(logits, T, E, tk, dev, out)
    st = load().fp8_moe_route(zp, T, E, ld, _OTYPES[logits.dtype], top_k, 1 if renorm else 0, mp, *ptrs, _stream())
    if st:
        _check("fp8_moe_route", st)
    return out


_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
_GROUP_SCORES = {"max": GROUP_MAX, "top2": GROUP_TOP2}


def _choice(name, value, choices):
    c = choices.get(value)
    if c is None:
        raise ValueError("%s: one of %s expected, got %r" % (name, ", ".join(choices), value))
    return c


def moe_route_grouped(logits, top_k, *, score="sigmoid", bias=None, groups=1, keep_groups=None, group_score="top2",
                      renorm=True, scale=1.0, mask=None, out: Optional[Routing] = None) -> Routing:
    """Routing of logits [T, E] (bf16 or fp32) by softmax or sigmoid scores: the
    top_k experts by score + bias (fp32 [E]) within the keep_groups best of
    `groups` runs of experts (all of them by default), by the largest value of a
    group ("max") or the sum of its two largest ("top2"); weights from the scores
    alone, times scale (see fp8_moe_route_grouped).  Routing's lse holds the
    scores' total; mask and `out` as in moe_route."""
    T, E = logits.shape
    dev, tk = _device(), (T, top_k)
    zp, ld = _mat("logits", logits, T, E, dev, _BF, _F32)
    mp = None if mask is None else _arr("mask", mask, (T,), dev, mask.dtype if mask.dtype is torch.bool else torch.uint8)
    bp = _arr("bias", bias, (E,), dev, _F32)
    out, ptrs = _routing(logits, T, E, tk, dev, out)
    st = load().fp8_moe_route_grouped(zp, T, E, ld, _OTYPES[logits.dtype], top_k, _choice("score", score, _SCORES), bp,
                                      groups, groups if keep_groups is None else keep_groups,
                                      _choice("group_score", group_score, _GROUP_SCORES), 1 if renorm else 0, scale, mp,
                                      *ptrs, _stream())
    if st:
        _check("fp8_moe_route_grouped", st)
    return out


def moe_route_grouped_backward(logits, experts, counts, total, *, dweights=None, dloss=None, score="sigmoid",
                               renorm=True, scale=1.0, out=None):
    """dlogits [T, E] (the logits' type) of sum(weights * dweights) + dloss . loss,
    from moe_route_grouped's outputs (total: its lse; see
    fp8_moe_route_grouped_backward)."""
    T, E = logits.shape
    dev, k, dt = _device(), experts.shape[1], logits.dtype
    zp, ld = _mat("logits", logits, T, E, dev, _BF, _F32)
    if out is None:
        out = torch.empty((T, E), dtype=dt, device=logits.device)
    op, ld_d = _mat("out", out, T, E, dev, dt)
    st = load().fp8_moe_route_grouped_backward(zp, T, E, ld, _OTYPES[dt], k, _choice("score", score, _SCORES),
                                               1 if renorm else 0, scale, _arr("experts", experts, (T, k), dev, _I32),
                                               _arr("counts", counts, (E + 1,), dev, _I32),
                                               _arr("total", total, (T,), dev, _F32),
                                               _arr("dweights", dweights, (T, k), dev, _F32),
                                               _arr("dloss", dloss, (2,), dev, _F32), op, ld_d, _stream())
    if st:
        _check("fp8_moe_route_grouped_backward", st)
    return out


def moe_bias_update(bias, counts, rate):
    """bias[e] += rate * sign(mean(counts) - counts[e]), in place: bias fp32 [E],
    counts int32 [E] or [E + 1] (moe_route_grouped's, whose last entry counts
    tokens)."""
    E, dev = bias.shape[0], _device()
    n = counts.shape[0]
    if n not in (E, E + 1):
        raise ValueError("counts: %d or %d numbers expected, got %d" % (E, E + 1, n))
    fp8_moe_bias_update(_arr("bias", bias, (E,), dev, _F32), _arr("counts", counts, (n,), dev, _I32), E, rate)
    return bias


def moe_route_backward(logits, experts, weights, counts, lse, *, dweights=None, dloss=None, renorm=True, out=None):
    """dlogits [T, E] (the logits' type) of sum(weights * dweights) +
    dloss . loss, from moe_route's outputs (see fp8_moe_route_backward)."""
    T, E = logits.shape
    dev, k, dt = _device(), experts.shape[1], logits.dtype
    tk = (T, k)
    zp, ld = _mat("logits", logits, T, E, dev, _BF, _F32)
    if out is None:
        out = torch.empty((T, E), dtype=dt, device=logits.device)
    op, ld_d = _mat("out", out, T, E, dev, dt)
    st = load().fp8_moe_route_backward(zp, T, E, ld, _OTYPES[dt], k, 1 if renorm else 0,
                                       _arr("experts", experts, tk, dev, _I32), _arr("weights", weights, tk, dev, _F32),
                                       _arr("counts", counts, (E + 1,), dev, _I32), _arr("lse", lse, (T,), dev, _F32),
                                       _arr("dweights", dweights, tk, dev, _F32), _arr("dloss", dloss, (2,), dev, _F32),
                                       op, ld_d, _stream())
    if st:
        _check("fp8_moe_route_backward", st)
    return out


def moe_combine_backward(dout, y, token_rows, weights, *, out=None):
    """(dy bf16 [rows, H], dweights fp32 [T, k]) of the combine, from dout
    [T, H] (bf16 or fp32) and the y [rows, H] it read.  Rows of dy without a
    slot are not written."""
    T, H = dout.shape
    dev, k, rows = _device(), token_rows.shape[1], y.shape[0]
    dop, ld_do = _mat("dout", dout, T, H, dev, _BF, _F32)
    yp, ld_y = _mat("y", y, rows, H, dev, _BF)
    if out is None:
        out = (torch.empty((rows, H), dtype=_BF, device=dout.device),
               torch.empty((T, k), dtype=_F32, device=dout.device))
    dy, dw = out
    dyp, ld_dy = _mat("out[0]", dy, rows, H, dev, _BF)
    st = load().fp8_moe_combine_backward(dop, ld_do, _OTYPES[dout.dtype], yp, rows, H, ld_y,
                                         _arr("token_rows", token_rows, (T, k), dev, _I32),
                                         _arr("weights", weights, (T, k), dev, _F32), T, k, dyp, ld_dy,
                                         _arr("out[1]", dw, (T, k), dev, _F32), _stream())
    if st:
        _check("fp8_moe_combine_backward", st)
    return out


# ------------------------------------------ linear layers in 8-bit integers
# Codes are int8 tensors whose rows are zero-padded to a multiple of 16 columns
# (the products' granularity along K) and scales fp32, one per row.
_I8 = torch.int8


def _pad16(n):
    return (n + 15) // 16 * 16


def i8_quant(x, axis: int = AXIS_ROW, out=None):
    """Codes and scales of a bf16 [rows, cols] tensor (see int8_quant): (q [rows,
    cols padded to 16], s [rows]), or with AXIS_COL the transposed codes with a
    scale per column, (q [cols, rows padded to 16], s [cols])."""
    rows, cols = x.shape
    dev = _device()
    xp, ld_x = _mat("x", x, rows, cols, dev, _BF)
    n, k = (rows, cols) if axis == AXIS_ROW else (cols, rows)
    if out is None:
        out = (torch.empty((n, _pad16(k)), dtype=_I8, device=x.device), torch.empty(n, dtype=_F32, device=x.device))
    qp, ld_q = _mat("out[0]", out[0], n, _pad16(k), dev, _I8)
    st = load().int8_quant(xp, rows, cols, ld_x, axis, qp, ld_q, _arr("out[1]", out[1], (n,), dev, _F32), _stream())
    if st:
        _check("int8_quant", st)
    return out


def i8_gemm(a, sa, b, sb, out_dtype=torch.bfloat16, out=None, ws=None):
    """C [M, N] = diag(sa) (A B^T) diag(sb) for int8 codes a [M, K], b [N, K] and
    fp32 scales sa [M], sb [N] (see int8_gemm).  ws: int8_gemm_ws_size bytes (uint8);
    made here where the call has use for it."""
    (M, K), N, dev = a.shape, b.shape[0], _device()
    ap, lda = _mat("a", a, M, K, dev, _I8)
    bp, ldb = _mat("b", b, N, K, dev, _I8)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    cp, ldc = _mat("out", out, M, N, dev, out_dtype)
    if ws is None:
        need = int8_gemm_ws_size(M, N, K)
        ws = _u8((need,), a.device) if need else None
    wsp, wsn = _workspace(ws, dev)
    st = load().int8_gemm(M, N, K, ap, lda, _arr("sa", sa, (M,), dev, _F32), bp, ldb, _arr("sb", sb, (N,), dev, _F32),
                          cp, ldc, _otype(out_dtype), wsp, wsn, _stream())
    if st:
        _check("int8_gemm", st)
    return out


class I8Linear(NamedTuple):
    """Output of i8_linear and its workspace."""
    y: torch.Tensor
    ws: torch.Tensor


def i8_linear(x, qw, sw, out_dtype=torch.bfloat16, out: Optional[I8Linear] = None) -> I8Linear:
    """Y = X W^T for X bf16 [rows, cols], quantized per token on the way, and a
    weight's codes qw [out features, cols padded to 16] and scales sw (i8_quant of
    the weight).  `out` is an earlier result for the same sizes whose tensors are
    written again (two calls in flight need two)."""
    (rows, cols), N, dev = x.shape, qw.shape[0], _device()
    xp, ld_x = _mat("x", x, rows, cols, dev, _BF)
    wp, ld_w = _mat("qw", qw, N, _pad16(cols), dev, _I8)
    if out is None:
        out = I8Linear(torch.empty((rows, N), dtype=out_dtype, device=x.device),
                       _u8((int8_linear_ws_size(rows, N, cols),), x.device))
    yp, ld_y = _mat("out.y", out.y, rows, N, dev, out_dtype)
    wsp, wsn = _workspace(out.ws, dev)
    st = load().int8_linear(rows, N, cols, xp, ld_x, wp, ld_w, _arr("sw", sw, (N,), dev, _F32), yp, ld_y,
                            _otype(out_dtype), wsp, wsn, _stream())
    if st:
        _check("int8_linear", st)
    return out


def i8_linear_forward(x, w, out_dtype=torch.bfloat16):
    """(y, saved) of a linear layer whose bf16 weight w [out, in] is quantized per
    output channel for this call; saved = (w, x) is what i8_linear_backward reads."""
    qw, sw = i8_quant(w)
    return i8_linear(x, qw, sw, out_dtype).y, (w, x)


class I8LinearGrads(NamedTuple):
    """Outputs of i8_linear_backward and its workspace."""
    dx: torch.Tensor
    dw: torch.Tensor
    ws: torch.Tensor


def i8_linear_backward(dy, saved, out: Optional[I8LinearGrads] = None) -> I8LinearGrads:
    """dX = dY W and dW = dY^T X, both fp32, of Y = X W^T in 8-bit integers, each
    operand with a scale per row of the product it enters: dY per token and W per
    input channel for dX, dY per output channel and X per input channel, both over
    the tokens, for dW (rounding to codes is passed straight through).  `out` is an
    earlier result for the same sizes whose tensors are written again (two calls in
    flight need two)."""
    w, x = saved
    (T, O), I, dev = dy.shape, x.shape[1], _device()
    dyp, ld_dy = _mat("dy", dy, T, O, dev, _BF)
    wp, ld_w = _mat("w", w, O, I, dev, _BF)
    xp, ld_x = _mat("x", x, T, I, dev, _BF)
    if out is None:
        e = lambda r, c: torch.empty((r, c), dtype=_F32, device=dy.device)
        out = I8LinearGrads(e(T, I), e(O, I), _u8((int8_linear_backward_ws_size(T, O, I),), dy.device))
    dxp, ld_dx = _mat("out.dx", out.dx, T, I, dev, _F32)
    dwp, ld_dw = _mat("out.dw", out.dw, O, I, dev, _F32)
    wsp, wsn = _workspace(out.ws, dev)
    st = load().int8_linear_backward(T, O, I, dyp, ld_dy, wp, ld_w, xp, ld_x, dxp, ld_dx, dwp, ld_dw, wsp, wsn, _stream())
    if st:
        _check("int8_linear_backward", st)
    return out


def i8_grouped_gemm(a, sa, b, sb, offsets, row_token=None, out_dtype=torch.bfloat16, out=None):
    """C [rows, N] of the experts' products (see int8_grouped_gemm): codes a [T, K]
    with scales sa [T], experts' codes b [G, N, K] with sb [G, N], int32 offsets
    [G + 1]; row r reads a's row row_token[r] (int32 [rows]; without it, row r).
    Rows from offsets[G] on are not written."""
    (T, K), (G, N, Kb), dev = a.shape, b.shape, _device()
    if Kb != K or b.dtype is not _I8 or b.get_device() != dev or (K > 1 and b.stride(2) != 1):
        raise ValueError("b: int8 [G, N, %d] with unit column stride on cuda:%d expected, got %s %s, strides %s, on %s"
                         % (K, dev, b.dtype, tuple(b.shape), b.stride(), b.device))
    ap, lda = _mat("a", a, T, K, dev, _I8)
    rows = T if row_token is None else row_token.numel()
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype, device=a.device)
    cp, ldc = _mat("out", out, rows, N, dev, out_dtype)
    st = load().int8_grouped_gemm(rows, N, K, G, _arr("offsets", offsets, (G + 1,), dev, _I32),
                                  _arr("row_token", row_token, (rows,), dev, _I32), T, ap, lda,
                                  _arr("sa", sa, (T,), dev, _F32), b.data_ptr(), b.stride(1) if N > 1 else K,
                                  b.stride(0) if G > 1 else 0, _arr("sb", sb, (G, N), dev, _F32), N, cp, ldc,
                                  _otype(out_dtype), _stream())
    if st:
        _check("int8_grouped_gemm", st)
    return out


def i8_silu_mul_quant(gate_up, live_rows=None, out=None):
    """Codes and scales of h = bf16(silu(gate) * up) per row, gate_up bf16 [rows,
    2 I] (see int8_silu_mul_quant): (q [rows, I padded to 16], s [rows]).
    live_rows: one int32 on the device; rows from it on are left alone."""
    rows, I, dev = gate_up.shape[0], gate_up.shape[1] // 2, _device()
    gp, ld = _mat("gate_up", gate_up, rows, 2 * I, dev, _BF)
    if out is None:
        out = (torch.empty((rows, _pad16(I)), dtype=_I8, device=gate_up.device),
               torch.empty(rows, dtype=_F32, device=gate_up.device))
    qp, ld_q = _mat("out[0]", out[0], rows, _pad16(I), dev, _I8)
    lp = None if live_rows is None else _arr("live_rows", live_rows, live_rows.shape, dev, _I32)
    if lp is not None and live_rows.numel() != 1:
        raise ValueError("live_rows: one number expected")
    st = load().int8_silu_mul_quant(gp, rows, I, ld, lp, qp, ld_q, _arr("out[1]", out[1], (rows,), dev, _F32), None, 0,
                                    _stream())
    if st:
        _check("int8_silu_mul_quant", st)
    return out


def i8_moe_forward(x, qgu, sgu, qdt, sdt, offsets, row_token, token_rows, weights, out_dtype=torch.bfloat16):
    """One MoE layer forward in 8-bit integers: X [T, H] per token, the experts'
    gate and up products (gathered by row_token), SiLU*mul and the codes of h, the
    down product, the routing-weighted combine over the slots that have a row.
    qgu [G, 2 I, H] codes (gate rows [0, I), up rows [I, 2 I)) with sgu [G, 2 I],
    qdt [G, H, I] with sdt [G, H]; H % 16 == I % 16 == 0.  offsets, row_token,
    token_rows and weights as moe_route and moe_route_grouped give them."""
    T, H = x.shape
    k, rows = token_rows.shape[1], row_token.numel()
    if H % 16 or qgu.shape[2] != H or qgu.shape[1] % 32 or qdt.shape != (qgu.shape[0], H, qgu.shape[1] // 2):
        raise ValueError("activations of %d columns, experts of %s and %s" % (H, tuple(qgu.shape), tuple(qdt.shape)))
    dev = _device()
    pos, w = _arr("token_rows", token_rows, (T, k), dev, _I32), _arr("weights", weights, (T, k), dev, _F32)
    qx, sx = i8_quant(x)
    gu = i8_grouped_gemm(qx, sx, qgu, sgu, offsets, row_token)
    qh, sh = i8_silu_mul_quant(gu, offsets[-1])
    y = i8_grouped_gemm(qh, sh, qdt, sdt, offsets)
    out = torch.empty((T, H), dtype=out_dtype, device=x.device)
    fp8_moe_combine_routed(y, rows, H, H, pos, w, T, k, out, H, _otype(out_dtype))
    return out


def gemm_splitk(a, sa, b, sb, bscale=BSCALE_BLOCK128, out_dtype=torch.bfloat16, splits=0):
    """gemm() with the K slices split among grid rows (splits 0: the
    planner's count); the fp32 workspace is allocated here with torch."""
    M, K = a.shape
    N = b.shape[0]
    out = OUT_FP32 if out_dtype == torch.float32 else OUT_BF16
    if splits == 0:
        splits, _ = fp8_blockscaled_gemm_splitk_plan(M, N, K, out)
    ws = torch.empty(max(splits, 1) * M * N if splits > 1 else 4, dtype=torch.float32, device=a.device)
    c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    fp8_blockscaled_gemm_splitk(M, N, K, a, a.stride(0), sa, sa.stride(0), sa.stride(1), b, b.stride(0), sb,
                                sb.stride(0), sb.stride(1), bscale, c, c.stride(0), out, splits, ws,
                                ws.numel() * 4)
    return c


def mx_quant(x: torch.Tensor):
    """MXFP8 1x32 quantization of bf16 [rows, cols] -> (q, s [rows, cols/32] uint8)."""
    rows, cols = x.shape
    q = _u8((rows, cols), x.device)
    s = _u8((rows, cols // 32), x.device)
    mxfp8_quant(x, rows, cols, x.stride(0), q, cols, s, cols // 32, 1)
    return q, s


def moe_combine(y: torch.Tensor, token_rows: torch.Tensor, weights: torch.Tensor, out_dtype=torch.bfloat16):
    """out[t] = sum_j weights[t, j] * y[token_rows[t, j]] for y bf16 [rows, H],
    token_rows int32 [T, k], weights fp32 [T, k]."""
    rows, H = y.shape
    T, k = token_rows.shape
    out = torch.empty((T, H), dtype=out_dtype, device=y.device)
    fp8_moe_combine(y, rows, H, y.stride(0), token_rows.contiguous(), weights.contiguous(), T, k, out, H,
                    OUT_FP32 if out_dtype == torch.float32 else OUT_BF16)
    return out


def mx_quant_t(x: torch.Tensor):
    """MXFP8 32x1 quantization along the rows of bf16 [rows, cols], written
    transposed -> (qt [cols, rows], s [cols, rows/32] uint8)."""
    rows, cols = x.shape
    qt = _u8((cols, rows), x.device)
    s = _u8((cols, rows // 32), x.device)
    mxfp8_quant_t(x, rows, cols, x.stride(0), qt, rows, s, rows // 32, 1)
    return qt, s


def mx_gemm(a, sa, b, sb, out_dtype=torch.float32):
    """Dense MXFP8 GEMM C = A B^T: a [M, K], b [N, K] codes, sa [M, K/32],
    sb [N, K/32] UE8M0 bytes (row-major)."""
    M, K = a.shape
    N = b.shape[0]
    c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    mxfp8_gemm(M, N, K, 0, None, None, M, a, a.stride(0), sa, sa.stride(0), b, b.stride(0), 0, sb, sb.stride(0), 0,
               c, N, OUT_FP32 if out_dtype == torch.float32 else OUT_BF16)
    return c


def quant_pow2(x: torch.Tensor, block_rows: int):
    """Power-of-two-scale quantization of bf16 [rows, cols] in 1x128
    (block_rows 1) or 128x128 (128) groups -> (q, s) with s a
    [row groups, ld_s] uint8 buffer, ld_s = 4 * ceil(cols / 512) (the GEMM's
    layout); s[:, :ceil(cols/128)] holds the bytes."""
    rows, cols = x.shape
    q = _u8((rows, cols), x.device)
    ld_s = 4 * ((cols + 511) // 512)
    s = torch.zeros(((rows + block_rows - 1) // block_rows, ld_s), dtype=torch.uint8, device=x.device)
    fp8_quant_pow2(x, rows, cols, x.stride(0), block_rows, q, cols, s, ld_s)
    return q, s


def gemm_pow2(a, sa, b, sb, out_dtype=torch.bfloat16):
    """C = A B^T with power-of-two scale bytes sa [M, lds_a], sb [N/128, lds_b]."""
    M, K = a.shape
    N = b.shape[0]
    c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    fp8_blockscaled_gemm_pow2(M, N, K, a, a.stride(0), sa, sa.stride(0), b, b.stride(0), sb, sb.stride(0), c, N,
                              OUT_FP32 if out_dtype == torch.float32 else OUT_BF16)
    return c


def e4m3_encode(v: torch.Tensor):
    out = _u8(v.shape, v.device)
    fp8bs_e4m3_encode(v.contiguous(), out, v.numel())
    return out
