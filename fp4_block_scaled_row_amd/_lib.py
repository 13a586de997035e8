"""ctypes loader for libfp4q.so (the C ABI declared in include/fp4q.h).

Argument marshalling only: every step of quantization runs in the HIP kernels
of the library.  There is no CPU fallback -- if the shared library is missing
or cannot be loaded, every call raises.
"""
import ctypes as C
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
# FP4Q_LIB selects another build of the same sources (the sanitizer run of the
# host-side tests loads a host-only AddressSanitizer/UBSan build this way)
LIB_PATH = os.environ.get("FP4Q_LIB") or os.path.join(HERE, "libfp4q.so")

FP4Q_OK, FP4Q_ERR_INVALID_ARG, FP4Q_ERR_UNSUPPORTED, FP4Q_ERR_WORKSPACE, FP4Q_ERR_NONFINITE, FP4Q_ERR_HIP = range(6)
FP4Q_F32, FP4Q_BF16, FP4Q_E4M3 = 0, 1, 2
FP4Q_MXFP4, FP4Q_NVFP4, FP4Q_IF4, FP4Q_MXFP8 = 0, 1, 2, 4
FP4Q_SCALE_OCP_MAX, FP4Q_SCALE_MANUAL, FP4Q_SCALE_NV_MAX6, FP4Q_SCALE_FOUR_OVER_SIX, FP4Q_SCALE_IF4 = 0, 1, 2, 3, 4
FP4Q_ROUND_RNE, FP4Q_ROUND_STOCHASTIC = 0, 1
FP4Q_ROT_NONE, FP4Q_ROT_FWHT_ROW, FP4Q_ROT_RHT16, FP4Q_ROT_FWHT128 = 0, 1, 2, 3
FP4Q_LINEAR, FP4Q_GATED, FP4Q_LINEAR_BACKWARD = 0, 1, 2

EXPORTED = [
    "fp4q_workspace_bytes", "fp4q_quantize_mxfp4", "fp4q_quantize_nvfp4", "fp4q_quantize_nvfp4_noalloc",
    "fp4q_silu_mul_fwht_mxfp4", "fp4q_fwht",
    "fp4q_dequantize", "fp4q_mxfp4_gemm",
    "fp4q_kv_write", "fp4q_kv_read", "fp4q_kv_attention", "fp4q_kv_attention_workspace_bytes",
    "fp4q_linear", "fp4q_gated", "fp4q_linear_backward", "fp4q_linear_workspace_bytes", "fp4q_gated_grad",
    "fp4q_rms_norm", "fp4q_rms_norm_backward", "fp4q_rms_norm_backward_workspace_bytes",
    "fp4q_check_counters", "fp4q_status_string", "fp4q_version",
]


class QuantArgs(C.Structure):
    _fields_ = [
        ("rows", C.c_int64), ("cols", C.c_int64), ("in_row_stride", C.c_int64),
        ("in_dtype", C.c_int32), ("block_size", C.c_int32), ("scale_policy", C.c_int32),
        ("manual_exponent", C.c_int32), ("rounding", C.c_int32), ("rotation", C.c_int32),
        ("seed", C.c_uint64),
    ]


class Outputs(C.Structure):
    _fields_ = [
        ("codes", C.c_void_p), ("scales", C.c_void_p), ("global_scale", C.c_void_p),
        ("choice_bits", C.c_void_p), ("rotated", C.c_void_p), ("counters", C.c_void_p),
    ]


class KvCacheArgs(C.Structure):
    _fields_ = [
        ("format", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("page_size", C.c_int32),
        ("num_pages", C.c_int64),
        ("k_codes", C.c_void_p), ("k_scales", C.c_void_p), ("v_codes", C.c_void_p), ("v_scales", C.c_void_p),
        ("k_global", C.c_void_p), ("v_global", C.c_void_p),
        ("code_stride", C.c_int64 * 3), ("scale_stride", C.c_int64 * 3),
    ]


class KvWriteArgs(C.Structure):
    _fields_ = [
        ("tokens", C.c_int64), ("k", C.c_void_p), ("v", C.c_void_p),
        ("k_stride", C.c_int64 * 2), ("v_stride", C.c_int64 * 2), ("slots", C.c_void_p),
        ("in_dtype", C.c_int32), ("rotation", C.c_int32),
    ]


class KvReadArgs(C.Structure):
    _fields_ = [
        ("page_table", C.c_void_p), ("table_stride", C.c_int64), ("table_cols", C.c_int32), ("seqs", C.c_int32),
        ("cu", C.c_void_p), ("starts", C.c_void_p), ("total", C.c_int64),
        ("k_out", C.c_void_p), ("v_out", C.c_void_p), ("out_dtype", C.c_int32), ("rotation", C.c_int32),
    ]


class KvAttentionArgs(C.Structure):
    _fields_ = [
        ("q", C.c_void_p), ("q_stride", C.c_int64 * 2), ("out", C.c_void_p), ("lse", C.c_void_p),
        ("cu_q", C.c_void_p), ("seq_lens", C.c_void_p), ("page_table", C.c_void_p), ("table_stride", C.c_int64),
        ("total_q", C.c_int64), ("table_cols", C.c_int32), ("seqs", C.c_int32), ("max_q", C.c_int32),
        ("q_heads", C.c_int32), ("dtype", C.c_int32), ("causal", C.c_int32), ("window", C.c_int32),
        ("rotation", C.c_int32), ("scale", C.c_float),
    ]


class WeightArgs(C.Structure):
    _fields_ = [
        ("format", C.c_int32), ("n", C.c_int64), ("k", C.c_int64),
        ("codes", C.c_void_p), ("scales", C.c_void_p), ("global_scale", C.c_void_p),
    ]


class LinearArgs(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("x_scales", C.c_void_p), ("rows", C.c_int64), ("x_stride", C.c_int64),
        ("x_dtype", C.c_int32), ("out_dtype", C.c_int32),
        ("bias", C.c_void_p), ("out", C.c_void_p), ("products", C.c_void_p), ("products_dtype", C.c_int32),
    ]


class GatedGradArgs(C.Structure):
    _fields_ = [
        ("dh", C.c_void_p), ("products", C.c_void_p), ("dproducts", C.c_void_p),
        ("rows", C.c_int64), ("f", C.c_int64), ("dh_stride", C.c_int64), ("dtype", C.c_int32),
        ("products_dtype", C.c_int32),
    ]


class RmsNormArgs(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("residual", C.c_void_p), ("x_stride", C.c_int64), ("residual_stride", C.c_int64),
        ("weight", C.c_void_p), ("y", C.c_void_p), ("summed", C.c_void_p), ("rstd", C.c_void_p),
        ("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64), ("d", C.c_int64),
        ("dtype", C.c_int32), ("weight_dtype", C.c_int32), ("eps", C.c_float),
    ]


class RmsNormGradArgs(C.Structure):
    _fields_ = [
        ("dy", C.c_void_p), ("s", C.c_void_p), ("ds", C.c_void_p),
        ("dy_stride", C.c_int64), ("s_stride", C.c_int64), ("ds_stride", C.c_int64),
        ("weight", C.c_void_p), ("rstd", C.c_void_p), ("dx", C.c_void_p), ("dw", C.c_void_p),
        ("rows", C.c_int64), ("d", C.c_int64), ("dtype", C.c_int32), ("weight_dtype", C.c_int32),
    ]


class Fp4qError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, status_string(status), status))


_lock = threading.Lock()
_lib = None


def load():
    """Load libfp4q.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfp4q.so is not built (run `python -m fp4_block_scaled_row_amd.build`); "
                               "there is no CPU fallback")
        lib = C.CDLL(LIB_PATH)
        vp, i64, i32, u64 = C.c_void_p, C.c_int64, C.c_int32, C.c_uint64
        lib.fp4q_workspace_bytes.argtypes = [C.POINTER(QuantArgs)]
        lib.fp4q_workspace_bytes.restype = C.c_size_t
        lib.fp4q_quantize_mxfp4.argtypes = [C.POINTER(QuantArgs), vp, C.POINTER(Outputs), vp, C.c_size_t, vp]
        lib.fp4q_quantize_mxfp4.restype = C.c_int
        lib.fp4q_quantize_nvfp4.argtypes = [C.POINTER(QuantArgs), vp, vp, C.POINTER(Outputs), vp, C.c_size_t, vp]
        lib.fp4q_quantize_nvfp4.restype = C.c_int
        lib.fp4q_quantize_nvfp4_noalloc.argtypes = [C.POINTER(QuantArgs), vp, vp, C.POINTER(Outputs), vp]
        lib.fp4q_quantize_nvfp4_noalloc.restype = C.c_int
        lib.fp4q_silu_mul_fwht_mxfp4.argtypes = [C.POINTER(QuantArgs), vp, vp, C.POINTER(Outputs), vp]
        lib.fp4q_silu_mul_fwht_mxfp4.restype = C.c_int
        lib.fp4q_fwht.argtypes = [i64, i64, i64, i32, vp, vp, i32, i32, u64, vp]
        lib.fp4q_fwht.restype = C.c_int
        lib.fp4q_dequantize.argtypes = [i32, i64, i64, i32, vp, vp, vp, i32, vp, vp]
        lib.fp4q_dequantize.restype = C.c_int
        lib.fp4q_mxfp4_gemm.argtypes = [i64, i64, i64, vp, vp, vp, vp, i32, vp, vp]
        lib.fp4q_mxfp4_gemm.restype = C.c_int
        kvp = C.POINTER(KvCacheArgs)
        lib.fp4q_kv_write.argtypes = [kvp, C.POINTER(KvWriteArgs), vp]
        lib.fp4q_kv_write.restype = C.c_int
        lib.fp4q_kv_read.argtypes = [kvp, C.POINTER(KvReadArgs), vp]
        lib.fp4q_kv_read.restype = C.c_int
        lib.fp4q_kv_attention_workspace_bytes.argtypes = [kvp, C.POINTER(KvAttentionArgs)]
        lib.fp4q_kv_attention_workspace_bytes.restype = C.c_size_t
        lib.fp4q_kv_attention.argtypes = [kvp, C.POINTER(KvAttentionArgs), vp, C.c_size_t, vp]
        lib.fp4q_kv_attention.restype = C.c_int
        wp, lp = C.POINTER(WeightArgs), C.POINTER(LinearArgs)
        for call in (lib.fp4q_linear, lib.fp4q_gated, lib.fp4q_linear_backward):
            call.argtypes = [wp, lp, vp, C.c_size_t, vp]
            call.restype = C.c_int
        lib.fp4q_linear_workspace_bytes.argtypes = [wp, lp, i32]
        lib.fp4q_linear_workspace_bytes.restype = C.c_size_t
        lib.fp4q_gated_grad.argtypes = [C.POINTER(GatedGradArgs), vp]
        lib.fp4q_gated_grad.restype = C.c_int
        lib.fp4q_rms_norm.argtypes = [C.POINTER(RmsNormArgs), vp]
        lib.fp4q_rms_norm.restype = C.c_int
        lib.fp4q_rms_norm_backward.argtypes = [C.POINTER(RmsNormGradArgs), vp, C.c_size_t, vp]
        lib.fp4q_rms_norm_backward.restype = C.c_int
        lib.fp4q_rms_norm_backward_workspace_bytes.argtypes = [C.POINTER(RmsNormGradArgs)]
        lib.fp4q_rms_norm_backward_workspace_bytes.restype = C.c_size_t
        lib.fp4q_check_counters.argtypes = [vp]
        lib.fp4q_check_counters.restype = C.c_int
        lib.fp4q_status_string.argtypes = [C.c_int]
        lib.fp4q_status_string.restype = C.c_char_p
        lib.fp4q_version.argtypes = []
        lib.fp4q_version.restype = C.c_char_p
        _lib = lib
        return lib


def status_string(status):
    return load().fp4q_status_string(int(status)).decode()


def check(status, where):
    if status != FP4Q_OK:
        raise Fp4qError(status, where)
