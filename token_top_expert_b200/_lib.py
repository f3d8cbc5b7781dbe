"""ctypes loader of libmsb.so (the C ABI declared in include/msb*.h).

Loading fails loudly: there is no fallback implementation of any step.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# MSB_VARIANT=instr selects the instrumented build (phase marks, wait-expiry injection)
VARIANT = os.environ.get("MSB_VARIANT") or None
LIB_PATH = os.path.join(_HERE, "libmsb_instr.so" if VARIANT == "instr" else "libmsb.so")

MSB_OK = 0
MSB_EINVAL = -1
MSB_EUNSUPPORTED = -2
MSB_ECUDA = -3
MSB_ETIMEOUT = -4
MSB_ENONFINITE = -5
MSB_EINTERNAL = -6
MSB_FLAG_GENERAL = 1
MSB_FLAG_X_READY = 2
MSB_FLAG_SINGLE = 4

MSB_MAX_D = 8192
MSB_MAX_INTER = 4096
MSB_MAX_EXPERTS = 512
MSB_MAX_TOP_E = 16
MSB_MAX_RANK = 128
MSB_MAX_BATCH = 256

# every function include/msb.h, msb_prep.h, msb_q4.h and msb_dense.h declare
SYMBOLS = (
    "msb_sketch_words", "msb_alpha_count", "msb_pack", "msb_ternary_rows", "msb_workspace_size",
    "msb_workspace_init", "msb_check", "msb_strerror", "moe_sparse_block",
    "moe_sparse_block_threshold", "msb_residual_rmsnorm", "msb_path_info",
    "moe_sparse_block_noalloc", "msb_noalloc_check", "moe_sparse_block_top_e",
    "moe_sparse_block_host",
    "msb_q4_record_bytes", "msb_pack_q4", "moe_sparse_block_q4",
    "msb_dense_check", "msb_route_workspace_size", "msb_route", "msb_grouped_matmul",
    "msb_grouped_swiglu", "msb_int8_quantize", "msb_int8_matmul", "msb_int8_swiglu",
    "msb_int8_linear_workspace_size", "msb_int8_linear",
    "msb_combine", "msb_block_norm", "msb_dense_workspace_size", "moe_dense_block",
    "moe_dense_block_int8",
)
MSB_Q4_GROUP = 64
MSB_BF16 = 0
MSB_F32 = 1
MSB_DENSE_MAX_TOKENS = 1048576
MSB_GROUPED_MAX_NK = 1048576
MSB_GROUPED_MAX_ROWS = 1 << 30
MSB_NORM_MAX_D = 16384
MSB_INT8_MAX_K = 131056


class MsbDims(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("inter", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("top_e", ctypes.c_int32), ("rank", ctypes.c_int32), ("renorm", ctypes.c_int32)]


class MsbTrace(ctypes.Structure):
    _fields_ = [("expert_ids", ctypes.c_void_p), ("expert_w", ctypes.c_void_p),
                ("sel", ctypes.c_void_p), ("sel_count", ctypes.c_void_p),
                ("union_count", ctypes.c_void_p), ("scores", ctypes.c_void_p)]


class MsbGroupWeights(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_group", ctypes.c_int64),
                ("stride_part", ctypes.c_int64), ("stride_n", ctypes.c_int64),
                ("stride_k", ctypes.c_int64)]


class MsbError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = _lib.msb_strerror(status).decode() if _lib is not None else str(status)
        super().__init__("%s failed: %s (status %d)" % (what or "msb call", msg, status))


_lib = None


def load() -> ctypes.CDLL:
    """Load libmsb.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("%s is not built; run `python -m token_top_expert_b200.build%s`"
                          % (LIB_PATH, " --instrumented" if VARIANT == "instr" else ""))
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, U32, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_float
    I64 = ctypes.c_int64
    dims_p = ctypes.POINTER(MsbDims)
    w_p = ctypes.POINTER(MsbGroupWeights)
    trace_p = ctypes.POINTER(MsbTrace)
    sig = {
        "msb_sketch_words": (SZ, [dims_p]),
        "msb_alpha_count": (SZ, [dims_p]),
        "msb_pack": (I32, [P, P, P, P, dims_p, P, P, P, P, I32]),
        "msb_ternary_rows": (I32, [P, I32, I32, P, P]),
        "msb_q4_record_bytes": (SZ, [dims_p]),
        "msb_pack_q4": (I32, [P, P, P, P, dims_p, P, P, P, P, I32]),
        "msb_workspace_size": (SZ, [dims_p, I32]),
        "msb_workspace_init": (I32, [P, SZ, P]),
        "msb_check": (I32, [P, P]),
        "msb_strerror": (ctypes.c_char_p, [I32]),
        "moe_sparse_block": (I32, [P, I32, P, P, P, P, I32, P, P, P, dims_p, P, SZ, trace_p, U32, P]),
        "moe_sparse_block_q4": (I32, [P, I32, P, P, P, P, I32, P, P, P, dims_p, P, SZ, trace_p, U32, P]),
        "moe_sparse_block_threshold": (I32, [P, I32, P, P, P, P, F32, P, P, P, dims_p, P, SZ,
                                             trace_p, P]),
        "msb_residual_rmsnorm": (I32, [P, P, P, I32, I32, F32, P]),
        "msb_path_info": (I32, [dims_p, I32, I32, U32, P]),
        "moe_sparse_block_noalloc": (I32, [P, P, P, P, P, I32, P, P, P, dims_p, trace_p, P]),
        "msb_noalloc_check": (I32, [P]),
        "moe_sparse_block_top_e": (I32, [P, I32, P, P, P, P, I32, I32, P, P, P, dims_p, P, SZ,
                                         trace_p, U32, P]),
        "moe_sparse_block_host": (I32, [P, P, I32, P, P, P, P, I32, P, P, P, P, dims_p, P, SZ,
                                        U32, P]),
        "msb_dense_check": (I32, [P]),
        "msb_route_workspace_size": (SZ, [I32, I32]),
        "msb_route": (I32, [P, I32, I64, P, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P]),
        "msb_grouped_matmul": (I32, [P, I64, I32, P, P, I32, I32, w_p, I32, I32, P, I32, I64, P]),
        "msb_grouped_swiglu": (I32, [P, I64, I32, P, P, I32, I32, w_p, I32, I32, P, I64, P]),
        "msb_int8_quantize": (I32, [P, I32, I64, I32, I32, P, I64, P, P]),
        "msb_int8_matmul": (I32, [P, I64, P, I32, P, P, I32, I32, w_p, P, I32, I32, P, I32, I64, P]),
        "msb_int8_swiglu": (I32, [P, I64, P, I32, P, P, I32, I32, w_p, P, I32, I32, P, I64, P]),
        "msb_int8_linear_workspace_size": (SZ, [I32, I32]),
        "msb_int8_linear": (I32, [P, I32, I64, I32, P, P, I32, I32, w_p, P, I32, I32, I32, P, I32, I64, P, SZ, P]),
        "msb_combine": (I32, [P, I32, I64, I32, P, P, I32, I32, I32, P, I64, P]),
        "msb_block_norm": (I32, [P, I32, I64, P, I32, I64, P, P, I32, I32, P, I32, I64, I64, F32, F32,
                                 F32, P, I64, P, I64, I32, I32, P]),
        "msb_dense_workspace_size": (SZ, [dims_p, I32, I32]),
        "moe_dense_block": (I32, [P, I32, P, P, P, P, dims_p, P, SZ, P]),
        "moe_dense_block_int8": (I32, [P, I32, P, P, P, P, P, P, P, dims_p, P, SZ, P]),
    }
    if VARIANT == "instr":
        sig["msb_debug_set_marks"] = (I32, [P])
        sig["msb_debug_inject"] = (I32, [U32, ctypes.c_uint64])
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib
