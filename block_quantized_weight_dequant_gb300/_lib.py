"""ctypes declarations for libbqgemv.so (include/bqgemv.h).

The library is loaded on first use; that use raises ImportError if the
library has not been built.  There is no CPU or PyTorch fallback for any
operation in this package.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbqgemv.so")

BQ_OK, BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_ALIGN, BQ_ERR_QTYPE, BQ_ERR_CUDA, BQ_ERR_DEVICE = range(7)
BQ_Q4_0, BQ_Q8_0, BQ_Q4_K = 2, 8, 12
BQ_F32, BQ_F16, BQ_BF16 = 0, 1, 30
BQ_VERIFY_MAX_ROWS = 6
BQ_PREFIX_MAX_GROUPS = 64
BQ_DEVERR_PAGE, BQ_DEVERR_LENGTH, BQ_DEVERR_SLOT, BQ_DEVERR_POOL = 0x100, 0x200, 0x400, 0x800
BQ_DEVERR_WAIT = 0x1000

BQ_OP_GEMV, BQ_OP_GATE_UP_SILU = 0, 1

# every extern "C" symbol of include/bqgemv.h
EXPORTS = ("bq_version", "bq_status_str", "bq_packed_bytes", "bq_quantize_pack", "bq_gemv_q8_0",
           "bq_gemv_q4_0", "bq_gemv_q4_k", "bq_gemv_gate_up_silu", "bq_gemv_verify", "bq_gemv_qkv_bias",
           "bq_gemv_f16", "bq_gemv_f16_f16out", "bq_device_status",
           "bq_tree_lanes", "bq_stream_workspace_bytes", "bq_stream_plan_create",
           "bq_stream_plan_launch", "bq_stream_plan_tune", "bq_stream_plan_launches",
           "bq_stream_plan_destroy", "bq_stream_run_noalloc", "bq_kv_block_tables",
           "bq_kv_shared_tables", "bq_kv_copy_pages", "bq_kv_compact", "bq_kv_append", "bq_kv_append_norm",
           "bq_paged_attention_workspace_bytes", "bq_paged_attention",
           "bq_paged_prefix_attention_workspace_bytes", "bq_paged_prefix_attention", "bq_sandwich_norm")
BQ_NOALLOC_MAX_OPS = 512


class BqOp(ctypes.Structure):
    """struct bq_op of include/bqgemv.h"""
    _fields_ = [("kind", ctypes.c_int32), ("stage", ctypes.c_int32), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64), ("W", ctypes.c_void_p), ("W_up", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("y", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


_I32, _I64, _VP, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class BqKvCache(ctypes.Structure):
    """bq_kv_cache of include/bqgemv.h"""
    _fields_ = ([(n, _I32) for n in ("type", "kv_heads", "head_dim", "page_size")]
                + [(n, _I64) for n in ("pages", "page_stride", "head_stride", "slot_stride")]
                + [(n, _VP) for n in ("k", "v", "k_scale", "v_scale")])


class BqKvTables(ctypes.Structure):
    """bq_kv_tables of include/bqgemv.h"""
    _fields_ = ([(n, _I32) for n in ("requests", "page_size", "table_width", "pool")]
                + [(n, _I64) for n in ("table_stride", "max_tokens")]
                + [(n, _VP) for n in ("lens", "new_lens", "table", "free_pages", "free_count", "slots",
                                      "positions", "starts", "lens_out", "free_count_out", "refused")])


class BqKvSharing(ctypes.Structure):
    """bq_kv_sharing of include/bqgemv.h"""
    _fields_ = [(n, _VP) for n in ("parents", "refs", "copy_src", "copy_dst", "copy_count")]


class BqKvCompactArgs(ctypes.Structure):
    """bq_kv_compact_args of include/bqgemv.h"""
    _fields_ = ([(n, _I32) for n in ("requests", "page_size", "table_width", "pool")]
                + [(n, _I64) for n in ("table_stride", "max_moves")]
                + [(n, _VP) for n in ("lens", "table", "free_pages", "refs", "copy_src", "copy_dst", "copy_count",
                                      "moved", "free_count_out")])


class BqKvAppendArgs(ctypes.Structure):
    """bq_kv_append_args of include/bqgemv.h"""
    _fields_ = ([(n, _I32) for n in ("dtype", "heads", "rot", "axes", "interleaved")]
                + [("sections", _I32 * 3), ("tokens", _I64)]
                + [(n, _VP) for n in ("k", "v", "q", "q_out")]
                + [(n, _I64) for n in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride",
                                       "q_token_stride", "q_head_stride", "q_out_token_stride",
                                       "q_out_head_stride")]
                + [("slots", _VP), ("positions", _VP), ("position_stride", _I64), ("freq", _VP)])


class BqKvNormArgs(ctypes.Structure):
    """bq_kv_norm_args of include/bqgemv.h"""
    _fields_ = [("q_gain", _VP), ("k_gain", _VP), ("eps", _F)]


class BqAttentionArgs(ctypes.Structure):
    """bq_attention_args of include/bqgemv.h"""
    _fields_ = ([(n, _I32) for n in ("dtype", "requests", "rows", "heads", "table_width")]
                + [("scale", _F)]
                + [(n, _I64) for n in ("table_stride", "q_row_stride", "q_head_stride", "out_row_stride",
                                       "out_head_stride")]
                + [(n, _VP) for n in ("q", "out", "table", "lens")])


class BqSandwichArgs(ctypes.Structure):
    """bq_sandwich_args of include/bqgemv.h"""
    _fields_ = ([("dtype", _I32), ("h_dtype", _I32), ("rows", _I64), ("width", _I64)]
                + [(n, _VP) for n in ("y", "h", "gate", "post", "pre", "h_out", "x")]
                + [(n, _I64) for n in ("y_stride", "h_stride", "gate_stride", "h_out_stride", "x_stride")]
                + [(n, _F) for n in ("alpha", "beta", "eps")])


class BQError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: bq status {status} ({status_str(status)})")


def _declare(lib):
    i64, i32, vp, fp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
    sig = {
        "bq_version": (i32, []),
        "bq_status_str": (ctypes.c_char_p, [i32]),
        "bq_packed_bytes": (i64, [i32, i64, i64]),
        "bq_quantize_pack": (i32, [i32, vp, i64, i64, vp, vp]),
        "bq_gemv_q8_0": (i32, [vp, vp, vp, i64, i64, vp]),
        "bq_gemv_q4_0": (i32, [vp, vp, vp, i64, i64, vp]),
        "bq_gemv_q4_k": (i32, [vp, vp, vp, i64, i64, vp]),
        "bq_gemv_gate_up_silu": (i32, [i32, vp, vp, vp, vp, fp, vp, i64, i64, vp]),
        "bq_gemv_verify": (i32, [i32, vp, vp, vp, i32, i64, i64, vp]),
        "bq_gemv_qkv_bias": (i32, [i32, vp, vp, vp, vp, i64, i64, vp]),
        "bq_gemv_f16": (i32, [vp, vp, vp, i64, i64, vp]),
        "bq_gemv_f16_f16out": (i32, [vp, vp, vp, i64, i64, vp]),
        "bq_device_status": (i32, [ctypes.POINTER(ctypes.c_uint), i32]),
        "bq_tree_lanes": (i32, [i64]),
        "bq_stream_workspace_bytes": (i64, [i32, i32]),
        "bq_stream_plan_create": (i32, [i32, ctypes.POINTER(BqOp), i32, vp, i64,
                                        ctypes.POINTER(vp)]),
        "bq_stream_plan_launch": (i32, [vp, vp]),
        "bq_stream_plan_tune": (i32, [vp, i32, vp]),
        "bq_stream_plan_launches": (i32, [vp]),
        "bq_stream_plan_destroy": (i32, [vp]),
        "bq_stream_run_noalloc": (i32, [i32, ctypes.POINTER(BqOp), i32, vp]),
        "bq_kv_block_tables": (i32, [ctypes.POINTER(BqKvTables), vp]),
        "bq_kv_shared_tables": (i32, [ctypes.POINTER(BqKvTables), ctypes.POINTER(BqKvSharing), vp]),
        "bq_kv_copy_pages": (i32, [ctypes.POINTER(vp), i32, vp, vp, vp, i64, vp]),
        "bq_kv_compact": (i32, [ctypes.POINTER(BqKvCompactArgs), vp]),
        "bq_kv_append": (i32, [ctypes.POINTER(BqKvCache), ctypes.POINTER(BqKvAppendArgs), vp]),
        "bq_kv_append_norm": (i32, [ctypes.POINTER(BqKvCache), ctypes.POINTER(BqKvAppendArgs),
                                    ctypes.POINTER(BqKvNormArgs), vp]),
        "bq_paged_attention_workspace_bytes": (i64, [ctypes.POINTER(BqKvCache),
                                                     ctypes.POINTER(BqAttentionArgs)]),
        "bq_paged_attention": (i32, [ctypes.POINTER(BqKvCache), ctypes.POINTER(BqAttentionArgs), vp, i64, vp]),
        "bq_paged_prefix_attention_workspace_bytes": (i64, [ctypes.POINTER(BqKvCache), ctypes.POINTER(BqAttentionArgs),
                                                            ctypes.POINTER(i32), ctypes.POINTER(i32), i32]),
        "bq_paged_prefix_attention": (i32, [ctypes.POINTER(BqKvCache), ctypes.POINTER(BqAttentionArgs),
                                            ctypes.POINTER(i32), ctypes.POINTER(i32), i32, vp, i64, vp]),
        "bq_sandwich_norm": (i32, [ctypes.POINTER(BqSandwichArgs), vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load(path=LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -m block_quantized_weight_dequant_gb300.build`"
            " (or __graft_entry__.build()); this package has no fallback without it")
    return _declare(ctypes.CDLL(path))


_LIB = None


def get():
    """The loaded library (loaded on first use; ImportError if not built)."""
    global _LIB
    if _LIB is None:
        _LIB = load()
    return _LIB


class _LazyLib:
    def __getattr__(self, name):
        fn = getattr(get(), name)
        self.__dict__[name] = fn  # found without this call from now on
        return fn


lib = _LazyLib()


def status_str(status):
    return get().bq_status_str(int(status)).decode()


def check(status, what):
    if status != BQ_OK:
        raise BQError(status, what)
