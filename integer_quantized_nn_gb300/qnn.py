"""Thin Python binding of libqnn.so (the C ABI in include/qnn.h).

Argument marshalling only: every function here forwards device pointers
(``tensor.data_ptr()``), host scalars and the current CUDA stream to the
function of the same name in the CUDA library and raises ``QnnError`` on a
non-OK status.  All device memory is allocated by the caller (with torch);
nothing here computes any part of the quantized path.  There is no fallback:
if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from . import build as _build

# ---- enums (mirror include/qnn.h) ------------------------------------------------
QNN_OK, QNN_ERR_INVALID_ARG, QNN_ERR_UNSUPPORTED, QNN_ERR_ALIGNMENT = 0, 1, 2, 3
QNN_ERR_OVERFLOW_RISK, QNN_ERR_CUDA, QNN_ERR_TIMEOUT = 4, 5, 6
DTYPES = {"s8": 0, "u8": 1, "s4": 2, "u4": 3, "s32": 4, "f32": 5, "f16": 6, "bf16": 7}
SCHEMES = {"sym": 0, "asym": 1, "pow2": 2}
EPI_MODES = {"requant": 0, "dequant": 1, "s32": 2}
ELTWISE_OPS = {"add": 0, "mul": 1, "relu": 2}
NORMS = {"none": 0, "rms": 1, "layer": 2}


class QnnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class QParams(ctypes.Structure):
    _fields_ = [("scheme", ctypes.c_int32), ("per_channel", ctypes.c_int32),
                ("axis", ctypes.c_int32), ("narrow_range", ctypes.c_int32),
                ("scale", ctypes.c_void_p), ("zero_point", ctypes.c_void_p),
                ("shift", ctypes.c_void_p)]


class Epilogue(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("relu", ctypes.c_int32), ("out_dt", ctypes.c_int32),
                ("z_out", ctypes.c_int32), ("zp_term", ctypes.c_void_p), ("M", ctypes.c_void_p),
                ("Bq", ctypes.c_void_p), ("D", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("res_dt", ctypes.c_int32),
                ("z_res", ctypes.c_int32), ("R", ctypes.c_float),
                ("ptf_shift", ctypes.c_void_p), ("ptf_max_shift", ctypes.c_int32),
                ("row_scale", ctypes.c_void_p)]


class ConvGeom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("N", "H", "W", "C", "OC", "FH", "FW", "pad_h", "pad_w", "stride_h", "stride_w", "layout")]

    @property
    def OH(self):
        return (self.H + 2 * self.pad_h - self.FH) // self.stride_h + 1

    @property
    def OW(self):
        return (self.W + 2 * self.pad_w - self.FW) // self.stride_w + 1


class W4Geom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "K", "group", "w_dt", "scale_dt")]


class BlockNorm(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("post", "pre")]
                + [(n, ctypes.c_float) for n in ("eps_post", "eps_pre", "res_scale", "block_scale")]
                + [(n, ctypes.c_void_p) for n in ("gamma_post", "beta_post", "gamma_pre", "beta_pre", "gate")]
                + [(n, ctypes.c_int64) for n in ("gate_rows", "ld_r", "ld_y", "ld_h")])


class KvGeom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "D", "page", "kv_dt")]


class KvSeqs(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("ld_table", ctypes.c_int64), ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32)]


_lib = None
_SYMBOLS = {}


def _declare(L):
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    c_int = ctypes.c_int
    sig = {
        "q_quantize": (c_int, [vp, vp, c_int, c_int, vp, vp, vp]),
        "q_dequantize": (c_int, [vp, c_int, vp, c_int, vp, vp, vp]),
        "qnn_gemm_packed_b_bytes": (sz, [c_int, c_int]),
        "qgemm_prepack_b": (c_int, [vp, c_int, c_int, vp, vp, vp]),
        "q_fold_epilogue": (c_int, [c_int, c_int, i32, vp, f32, vp, c_int, vp, f32, vp, vp, vp, vp, vp]),
        "qnn_gemm_workspace_bytes": (sz, [c_int, c_int]),
        "qgemm_s8": (c_int, [vp, c_int, vp, c_int, c_int, c_int, vp, vp, vp, vp, sz, vp]),
        "qgemm_pack_a": (c_int, [vp, c_int, c_int, c_int, vp, vp, sz, vp]),
        "qgemm_s8_packed": (c_int, [vp, c_int, vp, c_int, c_int, c_int, vp, vp, vp, vp]),
        "qgemm_s8_static_scratch": (c_int, [vp, c_int, vp, c_int, c_int, c_int, vp, vp, vp, vp]),
        "qnn_conv_packed_w_bytes": (sz, [vp, c_int]),
        "qconv_prepack_w": (c_int, [vp, c_int, vp, vp, vp, vp]),
        "qnn_conv_workspace_bytes": (sz, [vp, c_int]),
        "qconv_u4s4": (c_int, [vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "qconv_u8s8": (c_int, [vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "qconv_u8u8": (c_int, [vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "qconv_prepack_w_u8": (c_int, [vp, vp, vp, vp, vp, vp]),
        "q_log_int_softmax": (c_int, [vp, i64, i64, f32, c_int, vp, vp]),
        "q_attn_shift_v": (c_int, [vp, vp, i64, c_int, c_int, c_int, c_int, vp, vp]),
        "q_int_layernorm": (c_int, [vp, i64, c_int, vp, c_int, f32, vp, vp, vp, c_int, vp, vp]),
        "q_eltwise_s8": (c_int, [c_int, vp, vp, i64, f32, c_int, vp, vp]),
        "q_quantize_rows_dynamic": (c_int, [vp, i64, i64, c_int, vp, vp, vp]),
        "qgemm_prepack_b_u8": (c_int, [vp, vp, c_int, c_int, vp, vp, vp]),
        "qgemm_prepack_b_ptf": (c_int, [vp, vp, c_int, c_int, vp, vp, vp]),
        "qnn_gemm_zw_workspace_bytes": (sz, [c_int, c_int]),
        "qgemm_zw": (c_int, [vp, c_int, vp, vp, c_int, c_int, c_int, vp, vp, vp, vp, sz, vp]),
        "q_layout_nchw64": (c_int, [vp, c_int, c_int, c_int, c_int, c_int, c_int, vp, vp]),
        "qconv_prepack_w_u4": (c_int, [vp, vp, vp, vp, vp, vp]),
        "q_lis_attn_v": (c_int, [vp, f32, vp, i64, c_int, c_int, c_int, c_int, vp, vp]),
        "qnn_gemv_w4_packed_bytes": (sz, [vp]),
        "qgemv_prepack_w4": (c_int, [vp, vp, vp, vp, vp, vp]),
        "qgemv_w4": (c_int, [vp, c_int, i64, vp, vp, i64, vp, vp, c_int, i64, vp]),
        "q_block_norm": (c_int, [vp, c_int, vp, c_int, i64, c_int, vp, vp, vp, c_int, vp, vp]),
        "qnn_block_norm_backward_workspace_bytes": (sz, [i64, c_int, vp]),
        "q_block_norm_backward": (c_int, [vp, c_int, vp, c_int, i64, c_int] + [vp] * 11 + [sz, vp]),
        "qnn_kv_page_bytes": (sz, [vp]),
        "q_kv_write": (c_int, [vp, vp, c_int, i64, i64, vp, vp, vp]),
        "q_kv_read": (c_int, [vp, vp, c_int, i64, i64, vp, vp, vp]),
        "q_kv_keep": (c_int, [vp, vp, vp, i64, vp, vp]),
        "qnn_kv_attn_workspace_bytes": (sz, [vp, vp, c_int]),
        "q_kv_attn": (c_int, [vp, c_int, i64, c_int, vp, vp, f32, vp, c_int, vp, i64, vp, vp, sz, vp]),
        "qnn_status_string": (ctypes.c_char_p, [c_int]),
        "qnn_check_device_error": (c_int, [vp]),
        "qnn_selftest_wait_timeout": (c_int, [ctypes.c_uint64, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
        _SYMBOLS[name] = fn


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Loads libqnn.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if build_if_missing and not _build.up_to_date():
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"libqnn.so not found at {path}: build it with "
                               "integer_quantized_nn_gb300.build.build()")
        L = ctypes.CDLL(path)
        _declare(L)
        _lib = L
    return _lib


def status_string(status: int) -> str:
    load()
    return _SYMBOLS["qnn_status_string"](int(status)).decode()


def _check(status: int, what: str):
    if status != QNN_OK:
        raise QnnError(status, what)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _packed(t, size: int, what: str) -> Optional[int]:
    """The address of a tensor that the library reads as packed elements of `size` bytes (an int32
    tensor's, where that is 4): a slice of wider rows, or integers of another size, would be read as
    other numbers, which may well be valid ones."""
    if t is None:
        return None
    if t.element_size() != size or t.is_floating_point() or not t.is_contiguous():
        raise QnnError(QNN_ERR_INVALID_ARG, f"{what} must be contiguous, of {8 * size}-bit integers")
    return t.data_ptr()


def _nbytes(t) -> int:
    return int(t.numel()) * int(t.element_size())


_current_stream = None


def _stream(stream) -> Optional[int]:
    global _current_stream
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    if _current_stream is None:
        import torch
        # the handle alone: a torch.cuda.Stream object for it takes longer than the launch
        handle, device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
        _current_stream = lambda: handle(device())  # noqa: E731
    return _current_stream()


def _shape(shape):
    arr = (ctypes.c_int64 * len(shape))(*[int(s) for s in shape])
    return arr


def qparams(scheme="sym", scale=None, zero_point=None, shift=None, per_channel=False, axis=0,
            narrow_range=False) -> QParams:
    return QParams(SCHEMES[scheme], int(per_channel), int(axis), int(narrow_range), _ptr(scale),
                   _ptr(zero_point), _ptr(shift))


def q_quantize(x, q, q_dt: str, params: QParams, shape=None, stream=None):
    """x: fp32 device tensor; q: uint8/int8 device tensor holding the codes
    (4-bit: packed, last dimension halved).  shape: logical shape (default x.shape)."""
    shp = tuple(x.shape) if shape is None else tuple(shape)
    load()
    _check(_SYMBOLS["q_quantize"](_ptr(x), _ptr(q), DTYPES[q_dt], len(shp), _shape(shp),
                                  ctypes.byref(params), _stream(stream)), "q_quantize")


def q_dequantize(q, q_dt: str, x, params: QParams, shape=None, stream=None):
    shp = tuple(x.shape) if shape is None else tuple(shape)
    load()
    _check(_SYMBOLS["q_dequantize"](_ptr(q), DTYPES[q_dt], _ptr(x), len(shp), _shape(shp),
                                    ctypes.byref(params), _stream(stream)), "q_dequantize")


def qnn_gemm_packed_b_bytes(N: int, K: int) -> int:
    load()
    return int(_SYMBOLS["qnn_gemm_packed_b_bytes"](int(N), int(K)))


def qgemm_prepack_b(B, B_packed, colsum=None, stream=None):
    """B: int8 [N, K] device tensor; B_packed: uint8 device tensor of
    qnn_gemm_packed_b_bytes(N, K) bytes, 1024-byte aligned."""
    N, K = B.shape
    load()
    _check(_SYMBOLS["qgemm_prepack_b"](_ptr(B), int(N), int(K), _ptr(B_packed), _ptr(colsum),
                                       _stream(stream)), "qgemm_prepack_b")


def q_fold_epilogue(N, a_dt: str, z_a: int, colsum, s_a: float, s_w, s_o: float, bias=None,
                    zp_term=None, M=None, Bq=None, D=None, w_per_channel=True, stream=None):
    load()
    _check(_SYMBOLS["q_fold_epilogue"](int(N), DTYPES[a_dt], int(z_a), _ptr(colsum), float(s_a),
                                       _ptr(s_w), int(w_per_channel), _ptr(bias), float(s_o),
                                       _ptr(zp_term), _ptr(M), _ptr(Bq), _ptr(D), _stream(stream)),
           "q_fold_epilogue")


def epilogue(mode="requant", relu=False, out_dt="s8", z_out=0, zp_term=None, M=None, Bq=None,
             D=None, bias=None, residual=None, res_dt="s8", z_res=0, R=0.0, ptf_shift=None,
             ptf_max_shift=0, row_scale=None) -> Epilogue:
    return Epilogue(EPI_MODES[mode], int(relu), DTYPES[out_dt], int(z_out), _ptr(zp_term), _ptr(M),
                    _ptr(Bq), _ptr(D), _ptr(bias), _ptr(residual), DTYPES[res_dt], int(z_res),
                    float(R), _ptr(ptf_shift), int(ptf_max_shift), _ptr(row_scale))


def qnn_gemm_workspace_bytes(M: int, K: int) -> int:
    load()
    return int(_SYMBOLS["qnn_gemm_workspace_bytes"](int(M), int(K)))


def qgemm_s8(A, a_dt: str, B_packed, M: int, N: int, K: int, epi: Epilogue, C, C_s32=None,
             workspace=None, stream=None):
    """workspace: optional uint8 device tensor of at least
    qnn_gemm_workspace_bytes(M, K) bytes (the pre-pass path); None: no scratch."""
    load()
    ws_bytes = 0 if workspace is None else _nbytes(workspace)
    _check(_SYMBOLS["qgemm_s8"](_ptr(A), DTYPES[a_dt], _ptr(B_packed), int(M), int(N), int(K),
                                ctypes.byref(epi), _ptr(C), _ptr(C_s32), _ptr(workspace),
                                ctypes.c_size_t(ws_bytes), _stream(stream)),
           "qgemm_s8")


def qgemm_pack_a(A, a_dt: str, M: int, K: int, A_packed, ptf_shift=None, stream=None):
    """Re-encodes A into A_packed (uint8 device tensor of at least
    qnn_gemm_workspace_bytes(M, K) bytes) for qgemm_s8_packed."""
    load()
    _check(_SYMBOLS["qgemm_pack_a"](_ptr(A), DTYPES[a_dt], int(M), int(K), _ptr(ptf_shift),
                                    _ptr(A_packed), ctypes.c_size_t(_nbytes(A_packed)),
                                    _stream(stream)), "qgemm_pack_a")


def qgemm_s8_packed(A_packed, a_dt: str, B_packed, M: int, N: int, K: int, epi: Epilogue, C,
                    C_s32=None, stream=None):
    load()
    _check(_SYMBOLS["qgemm_s8_packed"](_ptr(A_packed), DTYPES[a_dt], _ptr(B_packed), int(M), int(N),
                                       int(K), ctypes.byref(epi), _ptr(C), _ptr(C_s32),
                                       _stream(stream)), "qgemm_s8_packed")


QNN_GEMM_STATIC_SCRATCH_BYTES = 32 << 20


def qgemm_s8_static_scratch(A, a_dt: str, B_packed, M: int, N: int, K: int, epi: Epilogue, C,
                            C_s32=None, stream=None):
    """qgemm_s8 for callers that cannot allocate at call time: the workspace is
    the library's fixed device array (QNN_GEMM_STATIC_SCRATCH_BYTES); calls
    that overlap in time race on it."""
    load()
    _check(_SYMBOLS["qgemm_s8_static_scratch"](_ptr(A), DTYPES[a_dt], _ptr(B_packed), int(M), int(N),
                                               int(K), ctypes.byref(epi), _ptr(C), _ptr(C_s32),
                                               _stream(stream)), "qgemm_s8_static_scratch")


LAYOUTS = {"nhwc": 0, "nchw": 1, "nchw64": 2}


def conv_geom(N, H, W, C, OC, FH, FW, pad=(1, 1), stride=(1, 1), layout="nhwc") -> ConvGeom:
    return ConvGeom(N, H, W, C, OC, FH, FW, pad[0], pad[1], stride[0], stride[1], LAYOUTS[layout])


def qnn_conv_packed_w_bytes(g: ConvGeom, w_dt: str = "s4") -> int:
    load()
    return int(_SYMBOLS["qnn_conv_packed_w_bytes"](ctypes.byref(g), DTYPES[w_dt]))


def qconv_prepack_w(W, w_dt: str, g: ConvGeom, W_packed, colsum=None, stream=None):
    load()
    _check(_SYMBOLS["qconv_prepack_w"](_ptr(W), DTYPES[w_dt], ctypes.byref(g), _ptr(W_packed),
                                       _ptr(colsum), _stream(stream)), "qconv_prepack_w")


def qconv_prepack_w_u4(W, z_w, g: ConvGeom, W_packed, colsum=None, stream=None):
    """u4 filters (packed nibbles, OHWI) with per-filter zero points z_w (int32 [OC])."""
    load()
    _check(_SYMBOLS["qconv_prepack_w_u4"](_ptr(W), _ptr(z_w), ctypes.byref(g), _ptr(W_packed), _ptr(colsum),
                                           _stream(stream)), "qconv_prepack_w_u4")


def qconv_prepack_w_u8(W, z_w, g: ConvGeom, W_packed, colsum=None, stream=None):
    """u8 filters (bytes, OHWI) with per-filter zero points z_w (int32 [OC]), for qconv_u8u8."""
    load()
    _check(_SYMBOLS["qconv_prepack_w_u8"](_ptr(W), _ptr(z_w), ctypes.byref(g), _ptr(W_packed), _ptr(colsum),
                                           _stream(stream)), "qconv_prepack_w_u8")


def qnn_conv_workspace_bytes(g: ConvGeom, in_dt: str = "u4") -> int:
    load()
    return int(_SYMBOLS["qnn_conv_workspace_bytes"](ctypes.byref(g), DTYPES[in_dt]))


def qconv_u4s4(I, z_in: int, W_packed, g: ConvGeom, epi: Epilogue, O, O_s32=None, workspace=None,
               stream=None):
    """workspace: optional uint8 device tensor of at least
    qnn_conv_workspace_bytes(g, "u4") bytes (the pre-pass + TMA path)."""
    load()
    ws_bytes = 0 if workspace is None else _nbytes(workspace)
    _check(_SYMBOLS["qconv_u4s4"](_ptr(I), int(z_in), _ptr(W_packed), ctypes.byref(g),
                                  ctypes.byref(epi), _ptr(O), _ptr(O_s32), _ptr(workspace),
                                  ctypes.c_size_t(ws_bytes), _stream(stream)),
           "qconv_u4s4")


def qconv_u8s8(I, z_in: int, W_packed, g: ConvGeom, epi: Epilogue, O, O_s32=None, workspace=None, stream=None):
    """workspace: optional uint8 device tensor of at least qnn_conv_workspace_bytes(g, "u8") bytes."""
    load()
    ws_bytes = 0 if workspace is None else _nbytes(workspace)
    _check(_SYMBOLS["qconv_u8s8"](_ptr(I), int(z_in), _ptr(W_packed), ctypes.byref(g),
                                  ctypes.byref(epi), _ptr(O), _ptr(O_s32), _ptr(workspace),
                                  ctypes.c_size_t(ws_bytes), _stream(stream)),
           "qconv_u8s8")


def qconv_u8u8(I, z_in: int, W_packed, g: ConvGeom, epi: Epilogue, O, O_s32=None, workspace=None, stream=None):
    """u8 activations x u8 filters prepacked by qconv_prepack_w_u8."""
    load()
    ws_bytes = 0 if workspace is None else _nbytes(workspace)
    _check(_SYMBOLS["qconv_u8u8"](_ptr(I), int(z_in), _ptr(W_packed), ctypes.byref(g),
                                  ctypes.byref(epi), _ptr(O), _ptr(O_s32), _ptr(workspace),
                                  ctypes.c_size_t(ws_bytes), _stream(stream)),
           "qconv_u8u8")


def qgemm_prepack_b_u8(B, z_w, B_packed, colsum=None, stream=None):
    """u8 weights [N, K] with per-channel zero points z_w (int32 [N])."""
    load()
    N, K = B.shape
    _check(_SYMBOLS["qgemm_prepack_b_u8"](_ptr(B), _ptr(z_w), N, K, _ptr(B_packed), _ptr(colsum), _stream(stream)),
           "qgemm_prepack_b_u8")


def qgemm_prepack_b_ptf(B, ptf_shift, B_packed, colsum=None, stream=None):
    """s8 weights [N, K] times 2^ptf_shift[k] (u8 [K], each 0..3) folded into the image."""
    load()
    N, K = B.shape
    _check(_SYMBOLS["qgemm_prepack_b_ptf"](_ptr(B), _ptr(ptf_shift), N, K, _ptr(B_packed), _ptr(colsum),
                                           _stream(stream)), "qgemm_prepack_b_ptf")


def qnn_gemm_zw_workspace_bytes(M: int, K: int) -> int:
    load()
    return int(_SYMBOLS["qnn_gemm_zw_workspace_bytes"](int(M), int(K)))


def qgemm_zw(A, a_dt: str, B_packed, z_w, M: int, N: int, K: int, epi: Epilogue, C, C_s32=None, workspace=None,
             stream=None):
    """qgemm_s8 for u8 weights with zero points (the run-time row-sum term)."""
    load()
    ws_bytes = 0 if workspace is None else _nbytes(workspace)
    _check(_SYMBOLS["qgemm_zw"](_ptr(A), DTYPES[a_dt], _ptr(B_packed), _ptr(z_w), int(M), int(N), int(K),
                                ctypes.byref(epi), _ptr(C), _ptr(C_s32), _ptr(workspace), ws_bytes, _stream(stream)),
           "qgemm_zw")


def q_log_int_softmax(x, rows: int, L: int, S: float, bits: int, code, stream=None):
    """Log-Int-Softmax of int32 rows x [rows, L] into u8 log2 codes (2^bits: masked)."""
    load()
    _check(_SYMBOLS["q_log_int_softmax"](_ptr(x), int(rows), int(L), float(S), int(bits), _ptr(code),
                                          _stream(stream)), "q_log_int_softmax")


def q_attn_shift_v(code, v, batch: int, Lq: int, Lk: int, d: int, bits: int, out, stream=None):
    """out[b, i, j] = sum_t 2^(2^bits - 1 - code[b, i, t]) v[b, t, j] (int32)."""
    load()
    _check(_SYMBOLS["q_attn_shift_v"](_ptr(code), _ptr(v), int(batch), int(Lq), int(Lk), int(d),
                                       int(bits), _ptr(out), _stream(stream)), "q_attn_shift_v")


def q_int_layernorm(x, rows: int, C: int, s: float, gamma, beta, out_scale, y, y_dt: str = "s8",
                    alpha=None, alpha_max: int = 0, stream=None):
    """Integer LayerNorm of s8 rows x [rows, C] with PTF factors alpha (u8 [C])."""
    load()
    _check(_SYMBOLS["q_int_layernorm"](_ptr(x), int(rows), int(C), _ptr(alpha), int(alpha_max), float(s),
                                        _ptr(gamma), _ptr(beta), _ptr(out_scale), DTYPES[y_dt], _ptr(y),
                                        _stream(stream)), "q_int_layernorm")


def q_eltwise_s8(op: str, a, b, n: int, M: float, out, relu: bool = False, stream=None):
    """Quantized elementwise add / mul / relu on s8 codes."""
    load()
    _check(_SYMBOLS["q_eltwise_s8"](ELTWISE_OPS[op], _ptr(a), _ptr(b), int(n), float(M), int(relu), _ptr(out),
                                     _stream(stream)), "q_eltwise_s8")


def q_quantize_rows_dynamic(x, rows: int, cols: int, q, scale, narrow: bool = False, stream=None):
    """Per-row scale max|x| / 127 and s8 codes."""
    load()
    _check(_SYMBOLS["q_quantize_rows_dynamic"](_ptr(x), int(rows), int(cols), int(narrow), _ptr(q), _ptr(scale),
                                                _stream(stream)), "q_quantize_rows_dynamic")


def q_layout_nchw64(src, to_nchw64: bool, N: int, H: int, W: int, C: int, dt: str, dst, stream=None):
    """NHWC <-> NCHW64 block permutation of packed codes."""
    load()
    _check(_SYMBOLS["q_layout_nchw64"](_ptr(src), int(bool(to_nchw64)), int(N), int(H), int(W), int(C), DTYPES[dt],
                                        _ptr(dst), _stream(stream)), "q_layout_nchw64")


def q_lis_attn_v(x, S: float, v, batch: int, Lq: int, Lk: int, d: int, bits: int, out, stream=None):
    """Log-Int-Softmax of int32 logits x and the shift product with v in one kernel."""
    load()
    _check(_SYMBOLS["q_lis_attn_v"](_ptr(x), float(S), _ptr(v), int(batch), int(Lq), int(Lk), int(d), int(bits),
                                     _ptr(out), _stream(stream)), "q_lis_attn_v")


def w4_geom(N: int, K: int, group: int, w_dt: str = "s4", scale_dt: str = "f32") -> W4Geom:
    return W4Geom(int(N), int(K), int(group), DTYPES[w_dt], DTYPES[scale_dt])


def qnn_gemv_w4_packed_bytes(g: W4Geom) -> int:
    load()
    return int(_SYMBOLS["qnn_gemv_w4_packed_bytes"](ctypes.byref(g)))


def qgemv_prepack_w4(W, scale, g: W4Geom, W_packed, zero_point=None, stream=None):
    """W: packed 4-bit codes [N, K/2]; scale: [N, ceil(K / group)] of the geometry's scale
    type; zero_point: int32 of the same shape for u4, None for s4; W_packed: uint8 device
    tensor of qnn_gemv_w4_packed_bytes(g) bytes, 128-byte aligned."""
    load()
    _check(_SYMBOLS["qgemv_prepack_w4"](_ptr(W), _ptr(scale), _ptr(zero_point), ctypes.byref(g), _ptr(W_packed),
                                        _stream(stream)), "qgemv_prepack_w4")


def qgemv_w4(x, x_dt: str, W_packed, g: W4Geom, M: int, y, y_dt: str, bias=None, ldx: int = 0, ldy: int = 0,
             stream=None):
    """y [M, N] = x [M, K] times the 4-bit weights; ldx, ldy: elements between rows (0: packed)."""
    load()
    _check(_SYMBOLS["qgemv_w4"](_ptr(x), DTYPES[x_dt], int(ldx), _ptr(W_packed), ctypes.byref(g), int(M),
                                _ptr(bias), _ptr(y), DTYPES[y_dt], int(ldy), _stream(stream)), "qgemv_w4")


def block_norm(post: str = "none", pre: str = "rms", eps_post: float = 1e-6, eps_pre: float = 1e-6, gamma_post=None,
               beta_post=None, gamma_pre=None, beta_pre=None, gate=None, gate_rows: int = 0, res_scale: float = 1.0,
               block_scale: float = 1.0, ld_r: int = 0, ld_y: int = 0, ld_h: int = 0) -> BlockNorm:
    """Holds the tensors' addresses only: keep the tensors alive as long as the struct is used."""
    return BlockNorm(NORMS[post], NORMS[pre], float(eps_post), float(eps_pre), float(res_scale), float(block_scale),
                     _ptr(gamma_post), _ptr(beta_post), _ptr(gamma_pre), _ptr(beta_pre), _ptr(gate), int(gate_rows),
                     int(ld_r), int(ld_y), int(ld_h))


def q_block_norm(r, r_dt: str, y, y_dt: str, rows: int, C: int, params: BlockNorm, r_out=None, h=None,
                 h_dt: str = None, h_scale=None, stream=None):
    """r_out = res_scale r + block_scale gate norm_post(y), h = norm_pre(r_out); h_dt: y_dt (the
    default) or "s8", with h_scale fp32 [rows]."""
    load()
    _check(_SYMBOLS["q_block_norm"](_ptr(r), DTYPES[r_dt], _ptr(y), DTYPES[y_dt], int(rows), int(C),
                                    ctypes.byref(params), _ptr(r_out), _ptr(h), DTYPES[h_dt or y_dt], _ptr(h_scale),
                                    _stream(stream)), "q_block_norm")


def qnn_block_norm_backward_workspace_bytes(rows: int, C: int, params: BlockNorm) -> int:
    load()
    return int(_SYMBOLS["qnn_block_norm_backward_workspace_bytes"](int(rows), int(C), ctypes.byref(params)))


def q_block_norm_backward(r_out, r_dt: str, y, y_dt: str, rows: int, C: int, params: BlockNorm, dh, dr_out, dr, dy,
                          workspace=None, dgate=None, dgamma_pre=None, dbeta_pre=None, dgamma_post=None,
                          dbeta_post=None, stream=None):
    """Gradients of q_block_norm; workspace: uint8 device tensor of
    qnn_block_norm_backward_workspace_bytes(rows, C, params) bytes, for the parameters' gradients."""
    load()
    _check(_SYMBOLS["q_block_norm_backward"](
        _ptr(r_out), DTYPES[r_dt], _ptr(y), DTYPES[y_dt], int(rows), int(C), ctypes.byref(params), _ptr(dh),
        _ptr(dr_out), _ptr(dr), _ptr(dy), _ptr(dgate), _ptr(dgamma_pre), _ptr(dbeta_pre), _ptr(dgamma_post),
        _ptr(dbeta_post), _ptr(workspace), 0 if workspace is None else _nbytes(workspace), _stream(stream)),
        "q_block_norm_backward")


def kv_geom(heads: int, D: int, page: int, kv_dt: str = "s8") -> KvGeom:
    return KvGeom(int(heads), int(D), int(page), DTYPES[kv_dt])


def qnn_kv_page_bytes(g: KvGeom) -> int:
    load()
    return int(_SYMBOLS["qnn_kv_page_bytes"](ctypes.byref(g)))


def kv_seqs(pages, table, lens, rows: int, tokens: int, starts=None) -> KvSeqs:
    """The sequences of a call: pages uint8 [num_pages, qnn_kv_page_bytes(g)], table int32
    [batch, most pages], lens int32 [batch], starts int32 [batch + 1] or None (`tokens` rows
    each); all contiguous.  Holds the tensors' addresses only: keep the tensors alive as long as it is used."""
    for t, n, what in ((lens, table.shape[0], "lens"), (starts, table.shape[0] + 1, "starts")):
        if t is not None and t.numel() < n:
            raise QnnError(QNN_ERR_INVALID_ARG, f"kv_seqs: {what} of a batch of {table.shape[0]} has {n} entries")
    return KvSeqs(_packed(pages, 1, "kv_seqs: pages"), int(pages.shape[0]), _packed(table, 4, "kv_seqs: table"),
                  int(table.shape[1]), _packed(lens, 4, "kv_seqs: lens"), _packed(starts, 4, "kv_seqs: starts"),
                  int(rows), int(table.shape[0]), int(tokens))


def q_kv_write(k, v, x_dt: str, g: KvGeom, seqs: KvSeqs, ld_k: int = 0, ld_v: int = 0, stream=None):
    """Quantizes k, v [rows, heads, D] into the cache; ld_k, ld_v: elements between rows (0: packed)."""
    load()
    _check(_SYMBOLS["q_kv_write"](_ptr(k), _ptr(v), DTYPES[x_dt], int(ld_k), int(ld_v), ctypes.byref(g),
                                  ctypes.byref(seqs), _stream(stream)), "q_kv_write")


def q_kv_read(k, v, x_dt: str, g: KvGeom, seqs: KvSeqs, ld_k: int = 0, ld_v: int = 0, stream=None):
    """The newest tokens' values into k, v [rows, heads, D]; either may be None."""
    load()
    _check(_SYMBOLS["q_kv_read"](_ptr(k), _ptr(v), DTYPES[x_dt], int(ld_k), int(ld_v), ctypes.byref(g),
                                 ctypes.byref(seqs), _stream(stream)), "q_kv_read")


def q_kv_keep(g: KvGeom, seqs: KvSeqs, keep, n_keep, stream=None):
    """keep: int32 [batch, most], ascending newest tokens of each sequence; n_keep: int32 [batch]; contiguous."""
    load()
    if keep.shape[0] < seqs.batch or n_keep.numel() < seqs.batch:
        raise QnnError(QNN_ERR_INVALID_ARG, f"q_kv_keep: keep and n_keep of a batch of {seqs.batch}")
    _check(_SYMBOLS["q_kv_keep"](ctypes.byref(g), ctypes.byref(seqs), _packed(keep, 4, "q_kv_keep: keep"),
                                 int(keep.shape[1]), _packed(n_keep, 4, "q_kv_keep: n_keep"), _stream(stream)),
           "q_kv_keep")


def qnn_kv_attn_workspace_bytes(g: KvGeom, seqs: KvSeqs, heads_q: int) -> int:
    load()
    return int(_SYMBOLS["qnn_kv_attn_workspace_bytes"](ctypes.byref(g), ctypes.byref(seqs), int(heads_q)))


def q_kv_attn(q, x_dt: str, heads_q: int, g: KvGeom, seqs: KvSeqs, scale: float, out, workspace, mask=None, lse=None,
              ld_q: int = 0, ld_out: int = 0, stream=None):
    """Attention of q [rows, heads_q, D] over the cache into out; mask: int32 [rows, words], contiguous, bits
    of the newest tokens that a row sees (None: up to itself); workspace: uint8 device tensor of
    qnn_kv_attn_workspace_bytes(g, seqs, heads_q) bytes; lse: fp32 [rows, heads_q], contiguous, or None."""
    load()
    if lse is not None and not lse.is_contiguous():
        raise QnnError(QNN_ERR_INVALID_ARG, "q_kv_attn: lse must be contiguous")
    _check(_SYMBOLS["q_kv_attn"](_ptr(q), DTYPES[x_dt], int(ld_q), int(heads_q), ctypes.byref(g), ctypes.byref(seqs),
                                 float(scale), _packed(mask, 4, "q_kv_attn: mask"),
                                 0 if mask is None else int(mask.shape[-1]), _ptr(out),
                                 int(ld_out), _ptr(lse), _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "q_kv_attn")


def qnn_check_device_error(stream=None) -> int:
    """Synchronises the stream; returns the status (does not raise)."""
    load()
    return int(_SYMBOLS["qnn_check_device_error"](_stream(stream)))


def qnn_selftest_wait_timeout(limit_ns: int, stream=None):
    load()
    _check(_SYMBOLS["qnn_selftest_wait_timeout"](int(limit_ns), _stream(stream)),
           "qnn_selftest_wait_timeout")
