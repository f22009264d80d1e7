"""Python binding of libtopk (ragged per-row top-K on GB300).

Argument marshalling only: every function here forwards to the C ABI declared
in ``include/libtopk.h`` with the same name; all computation runs in the CUDA
kernels of ``libtopk.so``. Tensor arguments may be torch tensors (their
``data_ptr()`` is passed) or raw integer device addresses. PyTorch serves only
as the provider of device memory and streams.

If ``libtopk.so`` has not been built this module raises on first use; there is
no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "TOPK_OK", "TopkError", "TopkOptions", "TopkDeviceProps", "TopkPlan",
    "topk_workspace_size", "topk_workspace_init", "topk_ragged", "topk_ragged_ex", "topk_ragged_static",
    "topk_ragged_strided", "topk_gather_sort",
    "topk_get_status", "topk_status_string", "topk_query_device", "topk_make_plan",
    "topk_kv_map", "topk_index_logits", "topk_paged_attention", "topk_attention_workspace_size",
    "TopkPagedRows", "TopkKvMapArgs", "TopkIndexLogitsArgs", "TopkAttentionArgs",
    "topk_block_means", "topk_block_scores", "topk_block_attention", "topk_shared_attention", "topk_shared_attention_scratch_size",
    "topk_page_fork", "topk_page_free", "topk_page_compact", "topk_page_copy",
    "TopkBlockMeansArgs", "TopkBlockScoresArgs", "TopkBlockAttentionArgs", "TopkSharedAttentionArgs", "TopkPagePool",
    "TopkPageForkArgs", "TopkPageFreeArgs", "TopkPageCompactArgs", "TopkPageCache", "TopkPageCopyArgs",
    "library_path", "Selector", "PagedDecoder", "KvMap", "PageCopies", "PageCaches",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libtopk.so")
_lock = threading.Lock()
_lib = None

TOPK_OK = 0
TOPK_ERR_INVALID_ARG = 1
TOPK_ERR_UNSUPPORTED_TOPK = 2
TOPK_ERR_MISALIGNED = 3
TOPK_ERR_WORKSPACE_TOO_SMALL = 4
TOPK_ERR_CUDA = 5
TOPK_ERR_BARRIER_TIMEOUT = 6
TOPK_ERR_LENGTH_CLAMPED = 7
TOPK_ERR_PLAN = 8
TOPK_ERR_UNSUPPORTED = 9

TOPK_MERGE_AUTO = 0
TOPK_MERGE_WORKSPACE = 1
TOPK_MERGE_CLUSTER = 2

TOPK_SHAPE_AUTO = 0
TOPK_SHAPE_WIDE = 1
TOPK_SHAPE_PAIR = 2
TOPK_SHAPE_SMALL = 3
TOPK_SHAPE_SHORT = 4

TOPK_DEV_LENGTH_CLAMPED = 0x1
TOPK_DEV_BARRIER_TIMEOUT = 0x2
TOPK_DEV_STAGE_TIMEOUT = 0x4
TOPK_DEV_WORKSPACE_DIRTY = 0x8
TOPK_DEV_BLOCKS_EXHAUSTED = 0x10
TOPK_DEV_TABLE_FULL = 0x20
TOPK_DEV_TOKENS_DROPPED = 0x40
TOPK_DEV_BAD_BLOCK = 0x80
TOPK_DEV_PIPELINE_TIMEOUT = 0x100

TOPK_DTYPE_F16 = 1
TOPK_DTYPE_BF16 = 2
TOPK_DTYPE_F8E4M3 = 3

TOPK_PAGED_WORKSPACE_BYTES = 256
TOPK_MAX_PAGE_CACHES = 256

EXPORTED = ("topk_workspace_size", "topk_workspace_init", "topk_ragged", "topk_ragged_ex", "topk_ragged_static",
            "topk_ragged_strided", "topk_gather_sort", "topk_get_status", "topk_status_string",
            "topk_query_device", "topk_make_plan", "topk_kv_map", "topk_index_logits", "topk_paged_attention",
            "topk_attention_workspace_size", "topk_block_means", "topk_block_scores", "topk_block_attention",
            "topk_shared_attention", "topk_shared_attention_scratch_size", "topk_page_fork", "topk_page_free",
            "topk_page_compact", "topk_page_copy")


class TopkError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {topk_status_string(code)} (code {code})")


class TopkOptions(ctypes.Structure):
    _fields_ = [("force_ctas_per_group", ctypes.c_int),
                ("long_row_threshold", ctypes.c_int64),
                ("barrier_timeout_us", ctypes.c_uint32),
                ("inject_skip_arrival", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t),
                ("max_ctas", ctypes.c_int),
                ("merge", ctypes.c_int),
                ("shape", ctypes.c_int),
                ("dependent_launch", ctypes.c_int)]


class TopkDeviceProps(ctypes.Structure):
    _fields_ = [("num_sms", ctypes.c_int),
                ("max_smem_optin", ctypes.c_int),
                ("smem_per_cta", ctypes.c_int),
                ("ctas_per_sm", ctypes.c_int),
                ("cluster_groups", ctypes.c_int * 9),
                ("pair_smem_per_cta", ctypes.c_int),
                ("pair_ctas_per_sm", ctypes.c_int),
                ("small_smem_per_cta", ctypes.c_int),
                ("small_ctas_per_sm", ctypes.c_int),
                ("short_smem_per_cta", ctypes.c_int),
                ("short_ctas_per_sm", ctypes.c_int),
                ("short_cluster_groups", ctypes.c_int * 9),
                ("short16_smem_per_cta", ctypes.c_int),
                ("short16_ctas_per_sm", ctypes.c_int),
                ("short16_cluster_groups", ctypes.c_int * 9)]


class TopkPlan(ctypes.Structure):
    _fields_ = [("ctas_per_group", ctypes.c_int),
                ("num_groups", ctypes.c_int),
                ("grid", ctypes.c_int),
                ("threads", ctypes.c_int),
                ("smem_bytes", ctypes.c_int),
                ("cooperative", ctypes.c_int),
                ("cluster", ctypes.c_int),
                ("shape", ctypes.c_int)]


class TopkPagedRows(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int64), ("next_n", ctypes.c_int), ("block_size", ctypes.c_int),
                ("num_requests", ctypes.c_int64), ("num_blocks", ctypes.c_int64), ("lengths", ctypes.c_void_p),
                ("row_request", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("max_blocks", ctypes.c_int64)]


class TopkKvMapArgs(ctypes.Structure):
    _fields_ = [("context_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("num_requests", ctypes.c_int64),
                ("block_size", ctypes.c_int), ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_blocks", ctypes.c_int64), ("free_blocks", ctypes.c_void_p), ("num_free", ctypes.c_int64),
                ("taken", ctypes.c_void_p), ("taken_out", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("row_lens", ctypes.c_void_p), ("row_request", ctypes.c_void_p), ("token_start", ctypes.c_void_p),
                ("max_tokens", ctypes.c_int64), ("workspace", ctypes.c_void_p)]


class TopkIndexLogitsArgs(ctypes.Structure):
    _fields_ = [("rows", TopkPagedRows), ("dtype", ctypes.c_int), ("heads", ctypes.c_int), ("dim", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("weights", ctypes.c_void_p), ("weight_row_stride", ctypes.c_int64), ("keys", ctypes.c_void_p),
                ("key_block_stride", ctypes.c_int64), ("key_token_stride", ctypes.c_int64),
                ("key_scales", ctypes.c_void_p), ("scale_block_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64), ("logits", ctypes.c_void_p),
                ("logits_row_stride", ctypes.c_int64), ("max_len", ctypes.c_int64), ("workspace", ctypes.c_void_p)]


class TopkAttentionArgs(ctypes.Structure):
    _fields_ = [("rows", TopkPagedRows), ("dtype", ctypes.c_int), ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("scale", ctypes.c_float), ("q", ctypes.c_void_p),
                ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("k_block_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v", ctypes.c_void_p), ("v_block_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64), ("indices", ctypes.c_void_p),
                ("index_row_stride", ctypes.c_int64), ("num_indices", ctypes.c_int), ("out", ctypes.c_void_p),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64), ("lse", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class TopkBlockMeansArgs(ctypes.Structure):
    _fields_ = [("context_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("num_requests", ctypes.c_int64),
                ("block_size", ctypes.c_int), ("dtype", ctypes.c_int), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("max_blocks", ctypes.c_int64), ("num_blocks", ctypes.c_int64),
                ("kv_heads", ctypes.c_int), ("dk", ctypes.c_int), ("k", ctypes.c_void_p),
                ("k_block_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("means", ctypes.c_void_p), ("mean_block_stride", ctypes.c_int64), ("mean_head_stride", ctypes.c_int64),
                ("workspace", ctypes.c_void_p)]


class TopkBlockScoresArgs(ctypes.Structure):
    _fields_ = [("rows", TopkPagedRows), ("dtype", ctypes.c_int), ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("dk", ctypes.c_int), ("sink_blocks", ctypes.c_int), ("recent_blocks", ctypes.c_int), ("q", ctypes.c_void_p),
                ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("means", ctypes.c_void_p),
                ("mean_block_stride", ctypes.c_int64), ("mean_head_stride", ctypes.c_int64), ("scores", ctypes.c_void_p),
                ("score_row_stride", ctypes.c_int64), ("score_head_stride", ctypes.c_int64),
                ("max_columns", ctypes.c_int64), ("score_lens", ctypes.c_void_p), ("workspace", ctypes.c_void_p)]


class TopkBlockAttentionArgs(ctypes.Structure):
    _fields_ = [("attention", TopkAttentionArgs), ("blocks", ctypes.c_void_p), ("block_row_stride", ctypes.c_int64),
                ("block_head_stride", ctypes.c_int64), ("num_chosen", ctypes.c_int64)]


class TopkSharedAttentionArgs(ctypes.Structure):
    _fields_ = [("attention", TopkAttentionArgs), ("prefix_of", ctypes.c_void_p), ("num_prefixes", ctypes.c_int64),
                ("prefix_lens", ctypes.c_void_p), ("prefix_table", ctypes.c_void_p), ("prefix_stride", ctypes.c_int64),
                ("prefix_blocks", ctypes.c_int64), ("scratch", ctypes.c_void_p), ("scratch_bytes", ctypes.c_size_t)]


class TopkPagePool(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("num_requests", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("max_blocks", ctypes.c_int64), ("shares", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("free_blocks", ctypes.c_void_p), ("num_free", ctypes.c_int64), ("taken", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p)]


class TopkPageForkArgs(ctypes.Structure):
    _fields_ = [("pool", TopkPagePool), ("parents", ctypes.c_void_p), ("children", ctypes.c_void_p),
                ("kept_lens", ctypes.c_void_p), ("num_forks", ctypes.c_int64), ("block_size", ctypes.c_int),
                ("source", ctypes.c_void_p), ("target", ctypes.c_void_p)]


class TopkPageFreeArgs(ctypes.Structure):
    _fields_ = [("pool", TopkPagePool), ("requests", ctypes.c_void_p), ("num_freed", ctypes.c_int64)]


class TopkPageCompactArgs(ctypes.Structure):
    _fields_ = [("pool", TopkPagePool), ("max_copies", ctypes.c_int64), ("source", ctypes.c_void_p),
                ("target", ctypes.c_void_p), ("block_table_out", ctypes.c_void_p), ("table_out_stride", ctypes.c_int64),
                ("shares_out", ctypes.c_void_p), ("free_blocks_out", ctypes.c_void_p), ("taken_out", ctypes.c_void_p),
                ("scratch", ctypes.c_void_p), ("scratch_bytes", ctypes.c_size_t)]


class TopkPageCache(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_stride", ctypes.c_int64),
                ("stride0", ctypes.c_int64), ("stride1", ctypes.c_int64), ("n0", ctypes.c_int32), ("n1", ctypes.c_int32),
                ("run_bytes", ctypes.c_int64)]


class TopkPageCopyArgs(ctypes.Structure):
    _fields_ = [("source", ctypes.c_void_p), ("target", ctypes.c_void_p), ("num_copies", ctypes.c_int64),
                ("caches", ctypes.c_void_p), ("num_caches", ctypes.c_int), ("workspace", ctypes.c_void_p)]


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m sparse_attention_row_gb300.build` "
                "(or __graft_entry__.build()); there is no fallback implementation")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.topk_workspace_size.restype = ctypes.c_size_t
        lib.topk_workspace_size.argtypes = [i32, i64, i64, i32, i32]
        lib.topk_workspace_init.restype = i32
        lib.topk_workspace_init.argtypes = [vp, ctypes.c_size_t, vp]
        lib.topk_ragged.restype = i32
        lib.topk_ragged.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, vp]
        lib.topk_ragged_ex.restype = i32
        lib.topk_ragged_ex.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, vp,
                                       ctypes.POINTER(TopkOptions)]
        lib.topk_ragged_strided.restype = i32
        lib.topk_ragged_strided.argtypes = [vp, i64, i64, i64, vp, i64, i32, i32, vp, vp, vp,
                                            ctypes.POINTER(TopkOptions)]
        lib.topk_gather_sort.restype = i32
        lib.topk_gather_sort.argtypes = [vp, i64, i64, i64, i64, i32, vp, vp, i32, vp]
        lib.topk_ragged_static.restype = i32
        lib.topk_ragged_static.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp]
        lib.topk_get_status.restype = i32
        lib.topk_get_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.topk_status_string.restype = ctypes.c_char_p
        lib.topk_status_string.argtypes = [i32]
        lib.topk_query_device.restype = i32
        lib.topk_query_device.argtypes = [i32, ctypes.POINTER(TopkDeviceProps)]
        lib.topk_make_plan.restype = i32
        lib.topk_make_plan.argtypes = [ctypes.POINTER(TopkDeviceProps), i64, i64, i32, i32,
                                       ctypes.POINTER(TopkOptions), ctypes.POINTER(TopkPlan)]
        for name in ("topk_kv_map", "topk_index_logits", "topk_paged_attention", "topk_block_means", "topk_block_scores",
                     "topk_block_attention", "topk_shared_attention", "topk_page_fork", "topk_page_free", "topk_page_compact",
                     "topk_page_copy"):
            getattr(lib, name).restype = i32
            getattr(lib, name).argtypes = [vp, vp]
        lib.topk_attention_workspace_size.restype = ctypes.c_size_t
        lib.topk_attention_workspace_size.argtypes = [i32]
        lib.topk_shared_attention_scratch_size.restype = ctypes.c_size_t
        lib.topk_shared_attention_scratch_size.argtypes = [i32, i64]
        _lib = lib
        return lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    raise TypeError(f"expected a tensor or an integer address, got {type(x).__name__}")


def _stream(stream) -> int | None:
    if stream is None:
        try:
            import torch

            if torch.cuda.is_available():
                return int(torch.cuda.current_stream().cuda_stream)
        except ImportError:
            pass
        return None
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def topk_status_string(code: int) -> str:
    return _load().topk_status_string(int(code)).decode()


def topk_workspace_size(device: int, num_rows: int = 0, row_stride: int = 1, next_n: int = 1,
                        topk: int = 2048) -> int:
    return int(_load().topk_workspace_size(device, num_rows, row_stride, next_n, topk))


def topk_workspace_init(workspace, nbytes: int, stream=None) -> int:
    return int(_load().topk_workspace_init(_ptr(workspace), nbytes, _stream(stream)))


def topk_ragged(logits, row_stride: int, lengths, num_rows: int, next_n: int, topk: int, out_idx,
                workspace, stream=None) -> int:
    return int(_load().topk_ragged(_ptr(logits), row_stride, _ptr(lengths), num_rows, next_n, topk,
                                   _ptr(out_idx), _ptr(workspace), _stream(stream)))


def topk_ragged_ex(logits, row_stride: int, lengths, num_rows: int, next_n: int, topk: int, out_idx,
                   workspace, stream=None, options: TopkOptions | None = None) -> int:
    opt = ctypes.byref(options) if options is not None else None
    return int(_load().topk_ragged_ex(_ptr(logits), row_stride, _ptr(lengths), num_rows, next_n,
                                      topk, _ptr(out_idx), _ptr(workspace), _stream(stream), opt))


def topk_ragged_strided(logits, row_stride: int, col_stride: int, max_len: int, lengths, num_rows: int,
                        next_n: int, topk: int, out_idx, workspace, stream=None,
                        options: TopkOptions | None = None) -> int:
    """topk_ragged over a strided view: element (r, i) at logits[r * row_stride + i * col_stride]."""
    opt = ctypes.byref(options) if options is not None else None
    return int(_load().topk_ragged_strided(_ptr(logits), row_stride, col_stride, max_len, _ptr(lengths),
                                           num_rows, next_n, topk, _ptr(out_idx), _ptr(workspace),
                                           _stream(stream), opt))


def topk_gather_sort(logits, row_stride: int, col_stride: int, max_len: int, num_rows: int, topk: int,
                     out_idx, out_val=None, sort: bool = True, stream=None) -> int:
    """Values of the selected indices (if out_val is given) and, with sort, rows ordered by
    value descending then index ascending, -1 last."""
    return int(_load().topk_gather_sort(_ptr(logits), row_stride, col_stride, max_len, num_rows, topk,
                                        _ptr(out_idx), _ptr(out_val), 1 if sort else 0, _stream(stream)))


def topk_ragged_static(logits, row_stride: int, lengths, num_rows: int, next_n: int, topk: int,
                       out_idx, stream=None) -> int:
    """topk_ragged for callers that cannot allocate: no workspace argument."""
    return int(_load().topk_ragged_static(_ptr(logits), row_stride, _ptr(lengths), num_rows, next_n,
                                          topk, _ptr(out_idx), _stream(stream)))


def topk_get_status(workspace, stream=None) -> tuple[int, int]:
    """Returns (code, device status bits); synchronises the stream."""
    word = ctypes.c_uint32(0)
    rc = _load().topk_get_status(_ptr(workspace), _stream(stream), ctypes.byref(word))
    return int(rc), int(word.value)


def topk_query_device(device: int) -> TopkDeviceProps:
    props = TopkDeviceProps()
    rc = _load().topk_query_device(device, ctypes.byref(props))
    if rc != TOPK_OK:
        raise TopkError(rc, "topk_query_device")
    return props


def topk_make_plan(props: TopkDeviceProps, num_rows: int, row_stride: int, next_n: int, topk: int,
                   options: TopkOptions | None = None) -> tuple[int, TopkPlan]:
    plan = TopkPlan()
    opt = ctypes.byref(options) if options is not None else None
    rc = _load().topk_make_plan(ctypes.byref(props), num_rows, row_stride, next_n, topk, opt,
                                ctypes.byref(plan))
    return int(rc), plan


def topk_kv_map(args: TopkKvMapArgs, stream=None) -> int:
    return int(_load().topk_kv_map(ctypes.byref(args), _stream(stream)))


def topk_index_logits(args: TopkIndexLogitsArgs, stream=None) -> int:
    return int(_load().topk_index_logits(ctypes.byref(args), _stream(stream)))


def topk_paged_attention(args: TopkAttentionArgs, stream=None) -> int:
    return int(_load().topk_paged_attention(ctypes.byref(args), _stream(stream)))


def topk_attention_workspace_size(device: int) -> int:
    return int(_load().topk_attention_workspace_size(device))


def topk_block_means(args: TopkBlockMeansArgs, stream=None) -> int:
    return int(_load().topk_block_means(ctypes.byref(args), _stream(stream)))


def topk_block_scores(args: TopkBlockScoresArgs, stream=None) -> int:
    return int(_load().topk_block_scores(ctypes.byref(args), _stream(stream)))


def topk_block_attention(args: TopkBlockAttentionArgs, stream=None) -> int:
    return int(_load().topk_block_attention(ctypes.byref(args), _stream(stream)))


def topk_shared_attention(args: TopkSharedAttentionArgs, stream=None) -> int:
    return int(_load().topk_shared_attention(ctypes.byref(args), _stream(stream)))


def topk_page_fork(args: TopkPageForkArgs, stream=None) -> int:
    return int(_load().topk_page_fork(ctypes.byref(args), _stream(stream)))


def topk_page_free(args: TopkPageFreeArgs, stream=None) -> int:
    return int(_load().topk_page_free(ctypes.byref(args), _stream(stream)))


def topk_page_compact(args: TopkPageCompactArgs, stream=None) -> int:
    return int(_load().topk_page_compact(ctypes.byref(args), _stream(stream)))


def topk_page_copy(args: TopkPageCopyArgs, stream=None) -> int:
    return int(_load().topk_page_copy(ctypes.byref(args), _stream(stream)))


def topk_shared_attention_scratch_size(device: int, num_rows: int) -> int:
    return int(_load().topk_shared_attention_scratch_size(device, num_rows))


class Selector:
    """Owns one workspace on one device and runs calls on a stream.

    Uses torch only to allocate the workspace and the output. Calls that may
    overlap on the GPU need separate Selectors (separate workspaces).
    """

    def __init__(self, device: int = 0):
        import torch

        self.device = device
        self.nbytes = topk_workspace_size(device)
        if self.nbytes == 0:
            raise TopkError(TOPK_ERR_CUDA, "topk_workspace_size")
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=f"cuda:{device}")
        rc = topk_workspace_init(self.workspace, self.nbytes)
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_workspace_init")

    def __call__(self, logits, lengths, topk: int, next_n: int | None = None, out=None, stream=None,
                 options: TopkOptions | None = None, sort: bool = False, values: bool = False):
        """Top-K indices of every row of a float32 [num_rows, max_len] tensor (any strides);
        with values=True also their values (returns (indices, values)), with sort=True each row
        ordered by value descending then index ascending, -1 last.

        lengths: int32, [num_rows], or [num_rows / next_n, next_n] for MTP, in which
        case next_n is taken from its second dimension (as the pages' launcher does).
        """
        import torch

        if logits.dtype != torch.float32 or logits.dim() != 2:
            raise ValueError("logits must be a float32 [num_rows, max_len] tensor")
        if lengths.dtype != torch.int32 or not lengths.is_contiguous() or lengths.dim() not in (1, 2):
            raise ValueError("lengths must be a contiguous int32 tensor with 1 or 2 dimensions")
        if next_n is None:
            next_n = lengths.shape[1] if lengths.dim() == 2 else 1
        num_rows, max_len = logits.shape
        if lengths.numel() != num_rows:
            raise ValueError("lengths must hold one length per row")
        if out is None:
            out = torch.empty((num_rows, topk), dtype=torch.int32, device=logits.device)
        # contiguous rows (stride(1) == 1) take the bulk-copy path inside the library
        rc = topk_ragged_strided(logits, logits.stride(0), logits.stride(1), max_len, lengths, num_rows,
                                 next_n, topk, out, self.workspace, stream, options)
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_ragged")
        if not (sort or values):
            return out
        val = torch.empty((num_rows, topk), dtype=torch.float32, device=logits.device) if values else None
        rc = topk_gather_sort(logits, logits.stride(0), logits.stride(1), max_len, num_rows, topk, out, val,
                              sort, stream)
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_gather_sort")
        return (out, val) if values else out

    def status(self, stream=None) -> int:
        rc, word = topk_get_status(self.workspace, stream)
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_get_status")
        return word

    def reset(self, stream=None) -> None:
        rc = topk_workspace_init(self.workspace, self.nbytes, stream)
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_workspace_init")


from .paged import KvMap, PageCaches, PageCopies, PagedDecoder  # noqa: E402
