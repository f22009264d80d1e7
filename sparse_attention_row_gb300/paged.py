"""The calls around the selection, for torch tensors: a paged cache's map, the
indexer's logits, attention over the cache (over chosen blocks of it, and over
prefixes that requests share), the blocks' means and scores, and the pages themselves.

Argument marshalling only, like the rest of the binding: shapes, strides and
types are read from the tensors, checked, and handed to ``libtopk.so``. A decode
step makes these calls back to back, so the checks are plain comparisons and the
arguments are packed in one go: a call with its outputs given is enqueued in 7 to 10 us of host time.
"""
from __future__ import annotations

import array
import struct
from typing import NamedTuple

import sparse_attention_row_gb300 as _sar

# The argument structs of include/libtopk.h in order, with native sizes and alignment
# (tests/test_paged_cpu.py compares them with the header's).
_ROWS = "qiiqqPPPqq"
_MAP = struct.Struct("@PPqiPqqPqPPPPPPqP")
_LOGITS = struct.Struct("@" + _ROWS + "iiiPqqPqPqqPqqPqqP")
_ATTEND = _ROWS + "iiiiifPqqPqqqPqqqPqiPqqPPN"
_POOL = "PqqqPqPqPP"
_ATTENTION = struct.Struct("@" + _ATTEND)
_MEANS = struct.Struct("@PPqiiPqqqiiPqqqPqqP")
_SCORES = struct.Struct("@" + _ROWS + "iiiiiiPqqPqqPqqqPP")
_BLOCKS = struct.Struct("@" + _ATTEND + "Pqqq")
_SHARED = struct.Struct("@" + _ATTEND + "PqPPqqPN")
_FORK = struct.Struct("@" + _POOL + "PPPqiPP")
_FREE = struct.Struct("@" + _POOL + "Pq")
_COMPACT = struct.Struct("@" + _POOL + "qPPPqPPPPN")
_CACHE = struct.Struct("@PqqqqiiQ")
_COPY = struct.Struct("@PPqPiP")


class KvMap(NamedTuple):
    """What ``PagedDecoder.kv_map`` lists for the new tokens of a step, packed request after request."""
    slots: "torch.Tensor"        # int64 [max_tokens], flat cache positions, -1 where there is none  # noqa: F821
    row_lens: "torch.Tensor"     # int32 [max_tokens], position + 1: the rows' lengths  # noqa: F821
    row_request: "torch.Tensor"  # int32 [max_tokens], -1 past the last token  # noqa: F821
    token_start: "torch.Tensor"  # int32 [requests + 1]  # noqa: F821


class PageCopies(NamedTuple):
    """Pages to copy: what ``PagedDecoder.fork_pages`` and ``compact_pages`` list and ``copy_pages`` does; -1 where there is nothing to copy."""
    source: "torch.Tensor"  # int32 [copies]  # noqa: F821
    target: "torch.Tensor"  # int32 [copies]  # noqa: F821


class PageCaches:
    """Caches whose pages are copied together, read once: made by ``PagedDecoder.page_caches``."""

    def __init__(self, tensors, packed: bytes, device: int):
        self.tensors, self.packed, self.device = tensors, array.array("B", packed), device
        self.address = self.packed.buffer_info()[0]


class PagedDecoder:
    """The paged calls on one device, with their workspace.

    Calls that may overlap on the GPU need separate PagedDecoders. ``stream`` is a torch
    stream (default: the current one); tensors that were made on another stream must be
    ready there, and outlive the call, as with any kernel, and so must the decoder with its
    workspace. Outputs made here belong to that stream. Making a decoder waits for the current
    stream, so that its workspace is cleared before a call on another.
    """

    def __init__(self, device: int = 0):
        import torch

        self._torch = torch
        self.device = device
        self._dev = torch.device("cuda", device)
        lib = _sar._load()
        self._kv_map, self._index_logits, self._attention = lib.topk_kv_map, lib.topk_index_logits, lib.topk_paged_attention
        self._block_means, self._block_scores, self._block_attention = lib.topk_block_means, lib.topk_block_scores, lib.topk_block_attention
        self._shared_attention = lib.topk_shared_attention
        self._fork, self._free, self._compact, self._copy = lib.topk_page_fork, lib.topk_page_free, lib.topk_page_compact, lib.topk_page_copy
        self._f32, self._i32, self._i64, self._u8 = torch.float32, torch.int32, torch.int64, torch.uint8
        self._scratch = {}  # bytes that shared_attention needs, by the number of rows
        self._dtypes = {torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}
        self._empty_tensor = torch.empty
        self._get_device, self._get_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.nbytes = _sar.topk_attention_workspace_size(device)
        if self.nbytes == 0:
            raise _sar.TopkError(_sar.TOPK_ERR_CUDA, "topk_attention_workspace_size")
        with torch.cuda.device(device):
            self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=self._dev)
            self._workspace_ptr = self.workspace.data_ptr()
            self.reset()
            # cleared before a first call on whichever stream (a capture runs nothing that could be waited for)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _on_stream(self, function, stream, *args):
        """function(*args, stream) with the decoder's device current, on the stream that its calls run on."""
        stream = self._get_stream(self.device) if stream is None else stream
        if self._get_device() == self.device:
            return function(*args, stream)
        with self._torch.cuda.device(self.device):
            return function(*args, stream)

    def reset(self, stream=None) -> None:
        """Clears the status word (stream-ordered)."""
        rc = self._on_stream(_sar.topk_workspace_init, stream, self.workspace, _sar.TOPK_PAGED_WORKSPACE_BYTES)
        if rc != _sar.TOPK_OK:
            raise _sar.TopkError(rc, "topk_workspace_init")

    def status(self, stream=None) -> int:
        """The sticky TOPK_DEV_* bits; synchronises the stream."""
        rc, word = self._on_stream(_sar.topk_get_status, stream, self.workspace)
        if rc != _sar.TOPK_OK:
            raise _sar.TopkError(rc, "topk_get_status")
        return word

    # Checks: each returns the tensor's address, and what else is wanted of it, or raises.

    def _bad(self, what: str, t, need: str):
        raise ValueError(f"{what} must be {need} on {self._dev}; got {tuple(t.shape)} {t.dtype}, strides {tuple(t.stride())}, on {t.device}")

    def _ints(self, what: str, t, n: int):
        """int32 [n], contiguous."""
        if t.dtype is not self._i32 or t.dim() != 1 or t.numel() != n or t.get_device() != self.device or not t.is_contiguous():
            self._bad(what, t, f"a contiguous int32 tensor with {n} entries")
        return t.data_ptr()

    def _matrix(self, what: str, t, dtype, rows: int):
        """[rows, any], rows contiguous: (address, row stride, columns)."""
        strides, shape = t.stride(), t.shape
        if len(strides) != 2 or t.dtype is not dtype or shape[0] != rows or t.get_device() != self.device or (strides[1] != 1 and shape[1] != 1):
            self._bad(what, t, f"a {dtype} tensor of {rows} contiguous rows")
        return t.data_ptr(), strides[0], shape[1]

    def _table(self, what: str, t):
        """int32 [rows, columns], rows contiguous: (address, rows, row stride, columns)."""
        strides, shape = t.stride(), t.shape
        if len(strides) != 2 or t.dtype is not self._i32 or t.get_device() != self.device or (strides[1] != 1 and shape[1] != 1):
            self._bad(what, t, "an int32 tensor of contiguous rows")
        rows, columns = shape
        stride = strides[0]
        return t.data_ptr(), rows, stride if rows > 1 or stride >= columns else columns, columns

    def _vectors(self, what: str, t, dtype, dims: int):
        """`dims` dimensions, the last one contiguous: (address, strides)."""
        strides = t.stride()
        if len(strides) != dims or t.dtype is not dtype or t.get_device() != self.device or (strides[-1] != 1 and t.shape[-1] != 1):
            self._bad(what, t, f"a {dims}-dimensional {dtype} tensor with a contiguous last dimension")
        return t.data_ptr(), strides

    def _cache(self, what: str, t, dtype):
        """[blocks, block_size, heads, dim] or, of one head, without that dimension: (address, strides of the first three, sizes)."""
        shape = t.shape
        if len(shape) == 3:
            p, (s0, s1, _) = self._vectors(what, t, dtype, 3)
            return p, s0, s1, 0, (shape[0], shape[1], 1), shape[2]
        p, (s0, s1, s2, _) = self._vectors(what, t, dtype, 4)
        blocks, block_size, heads, dim = shape
        return p, s0, s1, s2, (blocks, block_size, heads), dim

    def _empty(self, shape, dtype, stream):
        if stream is None:
            return self._empty_tensor(shape, dtype=dtype, device=self._dev)
        torch = self._torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self._dev)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self._dev)

    def _call(self, function, args: bytes, stream) -> None:
        if stream is None:
            stream = self._get_stream(self.device)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if self._get_device() == self.device:
            rc = function(args, stream)
        else:
            with self._torch.cuda.device(self.device):
                rc = function(args, stream)
        if rc != 0:
            raise _sar.TopkError(rc, function.__name__)

    def kv_map(self, context_lens, new_lens, block_table, free_blocks, taken, block_size: int, max_tokens: int,
               taken_out=None, out: KvMap | None = None, stream=None) -> KvMap:
        """Gives the requests' new tokens their places: enters the blocks taken from ``free_blocks`` in
        ``block_table`` (int32 [requests, columns], in place), advances ``taken`` (int32 [1]; into
        ``taken_out`` if that is given) and lists slot, length and request of every new token."""
        n = context_lens.numel()
        context, new = self._ints("context_lens", context_lens, n), self._ints("new_lens", new_lens, n)
        table, stride, columns = self._matrix("block_table", block_table, self._i32, n)
        free = free_blocks.numel()
        if out is None:  # four allocations, 6 us of host time; one, cut into views, takes 10
            out = KvMap(self._empty(max_tokens, self._i64, stream), self._empty(max_tokens, self._i32, stream),
                        self._empty(max_tokens, self._i32, stream), self._empty(n + 1, self._i32, stream))
            slots_ptr, lens_ptr, request_ptr, start_ptr = (x.data_ptr() for x in out)
        else:
            slots = out.slots
            if slots.dtype is not self._i64 or slots.dim() != 1 or slots.numel() != max_tokens or slots.get_device() != self.device or not slots.is_contiguous():
                self._bad("out.slots", slots, f"a contiguous int64 tensor with {max_tokens} entries")
            slots_ptr = slots.data_ptr()
            lens_ptr, request_ptr = self._ints("out.row_lens", out.row_lens, max_tokens), self._ints("out.row_request", out.row_request, max_tokens)
            start_ptr = self._ints("out.token_start", out.token_start, n + 1)
        taken_ptr = self._ints("taken", taken, 1)
        self._call(self._kv_map, _MAP.pack(
            context, new, n, block_size, table, stride if n > 1 or stride >= columns else columns, columns, self._ints("free_blocks", free_blocks, free), free, taken_ptr,
            taken_ptr if taken_out is None else self._ints("taken_out", taken_out, 1), slots_ptr, lens_ptr, request_ptr, start_ptr, max_tokens,
            self._workspace_ptr), stream)
        return out

    def _rows(self, rows: int, lengths, block_table, num_blocks: int, block_size: int, next_n, row_request):
        dims = lengths.dim()
        if lengths.dtype is not self._i32 or lengths.numel() != rows or (dims != 1 and dims != 2) or lengths.get_device() != self.device or not lengths.is_contiguous():
            self._bad("lengths", lengths, f"a contiguous int32 tensor with 1 or 2 dimensions and {rows} entries")
        if next_n is None:
            next_n = lengths.shape[1] if dims == 2 else 1
        table, requests, stride, columns = self._table("block_table", block_table)
        return (rows, next_n, block_size, requests, num_blocks, lengths.data_ptr(),
                0 if row_request is None else self._ints("row_request", row_request, rows), table, stride, columns)

    def index_logits(self, q, weights, keys, block_table, lengths, key_scales=None, next_n: int | None = None,
                     row_request=None, max_len: int | None = None, out=None, stream=None):
        """Scores of every cached token for every row: q [rows, heads, dim], weights fp32 [rows, heads],
        keys [blocks, block_size, dim] (fp16, bf16 or fp8 e4m3, as q), key_scales fp32 [blocks, block_size].
        Writes logits fp32 [rows, max_len] up to each row's length and leaves the rest of ``out`` as it is
        (what a new tensor holds there is undefined; the selection never uses it)."""
        rows, heads, dim = q.shape
        dtype = q.dtype
        kind = self._dtypes.get(dtype)
        if kind is None:
            raise ValueError(f"q has an unsupported type {dtype}")
        (qp, (q0, q1, _)), (kp, (k0, k1, _)) = self._vectors("q", q, dtype, 3), self._vectors("keys", keys, dtype, 3)
        wp, w0, weight_heads = self._matrix("weights", weights, self._f32, rows)
        blocks, block_size, key_dim = keys.shape
        if weight_heads != heads or key_dim != dim:
            raise ValueError("weights must have q's heads and keys its last dimension")
        sp, s0, s1 = 0, 0, 0
        if key_scales is not None:
            if key_scales.dtype is not self._f32 or key_scales.shape != keys.shape[:2] or key_scales.get_device() != self.device:
                self._bad("key_scales", key_scales, "a float32 [blocks, block_size] tensor")
            sp = key_scales.data_ptr()
            s0, s1 = key_scales.stride()
        rows_args = self._rows(rows, lengths, block_table, blocks, block_size, next_n, row_request)
        if out is None:
            out = self._empty((rows, block_table.shape[1] * block_size if max_len is None else max_len), self._f32, stream)
        op, o0, width = self._matrix("out", out, self._f32, rows)
        if max_len is not None:
            if max_len > width:
                raise ValueError("max_len must not exceed out's columns")
            width = max_len
        self._call(self._index_logits, _LOGITS.pack(
            *rows_args, kind, heads, dim, qp, q0, q1, wp, w0, kp, k0, k1, sp, s0, s1, op, o0, width, self._workspace_ptr), stream)
        return out

    def _attend(self, function, packer, more, q, k_cache, block_table, lengths, v_cache, v_dim, indices, scale, next_n, row_request, out, lse, return_lse, stream):
        """Checks an attention call's tensors and makes the call, `more` being its arguments behind them: (out, lse)."""
        rows, heads, dk = q.shape
        dtype = q.dtype
        kind = self._dtypes.get(dtype)
        if kind is None:
            raise ValueError(f"q has an unsupported type {dtype}")
        qp, (q0, q1, _) = self._vectors("q", q, dtype, 3)
        kp, k0, k1, k2, sizes, key_dim = self._cache("k_cache", k_cache, dtype)
        blocks, block_size, kv_heads = sizes
        if key_dim != dk:
            raise ValueError("q and k_cache must have the same last dimension")
        vp = v0 = v1 = v2 = 0
        if v_cache is not None:
            vp, v0, v1, v2, v_sizes, values = self._cache("v_cache", v_cache, dtype)
            if v_sizes != sizes or (v_dim is not None and v_dim != values):
                raise ValueError("v_cache must have k_cache's blocks and heads, and v_dim values")
            v_dim = values
        elif v_dim is None:
            raise ValueError("v_dim must be given where there is no v_cache")
        ip = i0 = topk = 0
        if indices is not None:
            ip, i0, topk = self._matrix("indices", indices, self._i32, rows)
        rows_args = self._rows(rows, lengths, block_table, blocks, block_size, next_n, row_request)
        if out is None:
            out = self._empty((rows, heads, v_dim), dtype, stream)
            op, o0, o1 = out.data_ptr(), heads * v_dim, v_dim
        else:
            op, (o0, o1, _) = self._vectors("out", out, dtype, 3)
            if out.shape != (rows, heads, v_dim):
                self._bad("out", out, f"a {(rows, heads, v_dim)} tensor")
        lp = 0
        if lse is not None:
            lp, _, lse_heads = self._matrix("lse", lse, self._f32, rows)
            if lse_heads != heads or not lse.is_contiguous():
                self._bad("lse", lse, f"a contiguous {(rows, heads)} tensor")
        elif return_lse:
            lse = self._empty((rows, heads), self._f32, stream)
            lp = lse.data_ptr()
        self._call(function, packer.pack(
            *rows_args, kind, heads, kv_heads, dk, v_dim, dk ** -0.5 if scale is None else scale, qp, q0, q1,
            kp, k0, k1, k2, vp, v0, v1, v2, ip, i0, topk, op, o0, o1, lp, self._workspace_ptr, self.nbytes, *more), stream)
        return out, lse

    def attention(self, q, k_cache, block_table, lengths, v_cache=None, v_dim: int | None = None, indices=None,
                  scale: float | None = None, next_n: int | None = None, row_request=None, out=None, lse=None,
                  return_lse: bool = False, stream=None):
        """Attention of q [rows, heads, dk] over a paged cache [blocks, block_size, kv_heads, dk] (or without
        the heads' dimension), over every token below each row's length or over ``indices``
        (int32 [rows, n], as the selection writes them). ``v_cache`` None: a token's value is the first
        ``v_dim`` elements of its key (latent attention). Returns out, or (out, lse)."""
        both = self._attend(self._attention, _ATTENTION, (), q, k_cache, block_table, lengths, v_cache, v_dim, indices, scale, next_n, row_request, out, lse, return_lse, stream)
        return both if return_lse else both[0]

    # ---- blocks chosen by a cheap score ----

    def block_means(self, k_cache, block_table, context_lens, new_lens, means, stream=None):
        """Brings ``means`` ([blocks, kv_heads, dk], of k_cache's type, in place) up to date after a step in which the requests
        got ``new_lens`` tokens behind ``context_lens`` (int32 [requests]): the mean key of every page that holds one of them."""
        dtype = k_cache.dtype
        kind = self._dtypes.get(dtype)
        if kind is None:
            raise ValueError(f"k_cache has an unsupported type {dtype}")
        kp, k0, k1, k2, (blocks, block_size, kv_heads), dk = self._cache("k_cache", k_cache, dtype)
        mp, (m0, m1, _) = self._vectors("means", means, dtype, 3)
        if means.shape != (blocks, kv_heads, dk):
            self._bad("means", means, f"a {(blocks, kv_heads, dk)} tensor")
        table, n, stride, columns = self._table("block_table", block_table)
        self._call(self._block_means, _MEANS.pack(
            self._ints("context_lens", context_lens, n), self._ints("new_lens", new_lens, n), n, block_size, kind, table, stride, columns, blocks, kv_heads, dk,
            kp, k0, k1, k2, mp, m0, m1, self._workspace_ptr), stream)
        return means

    def block_scores(self, q, means, block_table, lengths, block_size: int, sink_blocks: int = 0, recent_blocks: int = 0,
                     next_n: int | None = None, row_request=None, out=None, lens=None, stream=None):
        """Scores of every block (page) that a row sees, for each key-value head: the sum of the head's queries
        (q [rows, heads, dk]) times the page's mean key (``means`` [blocks, kv_heads, dk]); +inf for the first ``sink_blocks`` and the
        last ``recent_blocks``. Returns (fp32 [rows, kv_heads, columns], int32 [rows, kv_heads]: the blocks that each sees), which
        is what the selection takes: ``selector(scores.flatten(0, 1), lens.flatten(), n)``. Scores past them are left as they are.
        A row that is not its request's last one (of a prompt's piece, of drafted tokens) wants ``recent_blocks`` of 1 or more: its last block's
        mean holds tokens behind the row, and with 0 they take part in which blocks are selected."""
        rows, heads, dk = q.shape
        dtype = q.dtype
        kind = self._dtypes.get(dtype)
        if kind is None:
            raise ValueError(f"q has an unsupported type {dtype}")
        (qp, (q0, q1, _)), (mp, (m0, m1, _)) = self._vectors("q", q, dtype, 3), self._vectors("means", means, dtype, 3)
        blocks, kv_heads, mean_dim = means.shape
        if mean_dim != dk:
            raise ValueError("q and means must have the same last dimension")
        rows_args = self._rows(rows, lengths, block_table, blocks, block_size, next_n, row_request)
        if out is None:
            width = rows_args[-1]
            out = self._empty((rows, kv_heads, width), self._f32, stream)
            op, o0, o1 = out.data_ptr(), kv_heads * width, width
        else:
            op, (o0, o1, _) = self._vectors("out", out, self._f32, 3)
            out_rows, out_heads, width = out.shape
            if out_rows != rows or out_heads != kv_heads:
                self._bad("out", out, f"a {(rows, kv_heads)} x columns tensor")
        if lens is None:
            lens = self._empty((rows, kv_heads), self._i32, stream)
            lp = lens.data_ptr()
        else:
            lp, _, lens_heads = self._matrix("lens", lens, self._i32, rows)
            if lens_heads != kv_heads or not lens.is_contiguous():
                self._bad("lens", lens, f"a contiguous {(rows, kv_heads)} tensor")
        self._call(self._block_scores, _SCORES.pack(
            *rows_args, kind, heads, kv_heads, dk, sink_blocks, recent_blocks, qp, q0, q1, mp, m0, m1, op, o0, o1, width, lp, self._workspace_ptr), stream)
        return out, lens

    def block_attention(self, q, k_cache, block_table, lengths, blocks, v_cache=None, v_dim: int | None = None, scale: float | None = None,
                        next_n: int | None = None, row_request=None, out=None, lse=None, return_lse: bool = False, stream=None):
        """``attention`` over the tokens of chosen blocks: ``blocks`` int32 [rows, kv_heads, n], a list for each key-value head, or
        [rows, n], one for all heads of a row; columns of the row's request in the table, -1 where there is none."""
        shape = blocks.shape
        by_head = len(shape) != 2
        bp, strides = self._vectors("blocks", blocks, self._i32, 3 if by_head else 2)
        rows, kv_heads = q.shape[0], k_cache.shape[2] if by_head and k_cache.dim() == 4 else 1
        if shape[0] != rows or (by_head and shape[1] != kv_heads):
            self._bad("blocks", blocks, f"a {(rows, kv_heads)} x n or {rows} x n tensor")
        more = bp, strides[0], strides[1] if by_head else 0, shape[-1]
        both = self._attend(self._block_attention, _BLOCKS, more, q, k_cache, block_table, lengths, v_cache, v_dim, None, scale, next_n, row_request, out, lse, return_lse, stream)
        return both if return_lse else both[0]

    # ---- a prefix that requests share ----

    def shared_attention(self, q, k_cache, block_table, lengths, prefix_of, prefix_lens, prefix_table, v_cache=None, v_dim: int | None = None,
                         scale: float | None = None, next_n: int | None = None, row_request=None, out=None, lse=None,
                         return_lse: bool = False, stream=None):
        """``attention`` over everything cached, for requests of which some begin with the same pages: request b with the first
        ``prefix_lens[prefix_of[b]]`` tokens of the pages in ``prefix_table[prefix_of[b]]`` (int32 [requests], negative: nothing shared;
        [prefixes]; [prefixes, columns]). Their whole pages are read once for all neighbouring rows that begin with them. Lengths count the
        prefix, and the rows of ``block_table`` have its pages' columns. A request of which one of its ``next_n`` rows sees less than those
        pages hold reads its own row of the table; with ``row_request`` that goes for each such row by itself. How the call is done depends on
        ``prefix_table``'s width: give it the columns that the longest prefix needs, not more, where prefixes are short."""
        table, prefixes, stride, columns = self._table("prefix_table", prefix_table)
        rows = q.shape[0]
        need = self._scratch.get(rows)
        if need is None:
            need = self._scratch[rows] = _sar.topk_shared_attention_scratch_size(self.device, rows)
        scratch = self._empty(need, self._u8, stream)
        more = (self._ints("prefix_of", prefix_of, block_table.shape[0]), prefixes, self._ints("prefix_lens", prefix_lens, prefixes), table, stride, columns,
                scratch.data_ptr(), need)
        both = self._attend(self._shared_attention, _SHARED, more, q, k_cache, block_table, lengths, v_cache, v_dim, None, scale, next_n, row_request, out, lse, True, stream)
        return both if return_lse else both[0]

    # ---- the pages ----

    def _pool(self, block_table, shares, free_blocks, taken):
        blocks, free = shares.numel(), free_blocks.numel()
        table, requests, stride, columns = self._table("block_table", block_table)
        return (table, requests, stride, columns, self._ints("shares", shares, blocks), blocks, self._ints("free_blocks", free_blocks, free), free,
                self._ints("taken", taken, 1), self._workspace_ptr)

    def _copies(self, out, n: int, stream):
        if out is None:
            source, target = self._empty(n, self._i32, stream), self._empty(n, self._i32, stream)
            return PageCopies(source, target), source.data_ptr(), target.data_ptr()
        return out, self._ints("out.source", out.source, n), self._ints("out.target", out.target, n)

    def fork_pages(self, parents, children, kept_lens, block_table, shares, free_blocks, taken, block_size: int,
                   out: PageCopies | None = None, stream=None) -> PageCopies:
        """Gives each of ``children`` (rows of the table, int32) the first ``kept_lens`` tokens of its parent: it shares the parent's whole
        pages (``shares``: int32 [blocks], holders beyond the first), and gets a page of its own from ``free_blocks`` for what is left
        (``taken`` advances, as in ``kv_map``). Returns the copies into those, for ``copy_pages``. All in place; free what a child holds first."""
        n = parents.numel()
        pool = self._pool(block_table, shares, free_blocks, taken)
        out, source, target = self._copies(out, n, stream)
        self._call(self._fork, _FORK.pack(*pool, self._ints("parents", parents, n), self._ints("children", children, n), self._ints("kept_lens", kept_lens, n), n, block_size, source, target), stream)
        return out

    def free_pages(self, requests, block_table, shares, free_blocks, taken, stream=None) -> None:
        """Takes the pages of ``requests`` (rows of the table, int32) back, in place: those that no other row holds are put in front of
        the free ones (``taken`` goes down), in the order of requests and columns; the rows are set to -1."""
        n = requests.numel()
        self._call(self._free, _FREE.pack(*self._pool(block_table, shares, free_blocks, taken), self._ints("requests", requests, n), n), stream)

    def compact_pages(self, block_table, shares, free_blocks, taken, max_copies: int, table_out=None, shares_out=None, free_out=None,
                      taken_out=None, out: PageCopies | None = None, stream=None) -> PageCopies:
        """Moves the highest pages that the table names to the lowest free numbers, ``max_copies`` of them at most, and sorts the free
        ones. In place, or into the tensors that are given; tables made from this one (prefixes') are not renamed. Returns the moves;
        ``copy_pages`` brings the contents over."""
        pool = self._pool(block_table, shares, free_blocks, taken)
        requests, columns, blocks, free = pool[1], pool[3], pool[5], pool[7]
        table, stride = pool[0], pool[2]
        if table_out is not None:
            table, tall, stride, wide = self._table("table_out", table_out)
            if tall != requests or wide != columns:
                self._bad("table_out", table_out, f"a {(requests, columns)} tensor")
        out, source, target = self._copies(out, max_copies, stream)
        need = 12 * blocks + 16
        scratch = self._empty(need, self._u8, stream)
        self._call(self._compact, _COMPACT.pack(
            *pool, max_copies, source, target, table, stride, pool[4] if shares_out is None else self._ints("shares_out", shares_out, blocks),
            pool[6] if free_out is None else self._ints("free_out", free_out, free), pool[8] if taken_out is None else self._ints("taken_out", taken_out, 1),
            scratch.data_ptr(), need), stream)
        return out

    def page_caches(self, caches) -> PageCaches:
        """Reads caches ([blocks, ...] each, any type and strides whose pages are at most two loops over runs of bytes) for ``copy_pages``, to be
        kept by programs that copy among the same ones again."""
        caches = list(caches)
        if len(caches) > _sar.TOPK_MAX_PAGE_CACHES:
            raise ValueError(f"at most {_sar.TOPK_MAX_PAGE_CACHES} caches at a time")
        return PageCaches(caches, b"".join([self._page_cache(t) for t in caches]), self.device)

    def _page_cache(self, t) -> bytes:
        shape = t.shape
        if not shape or t.get_device() != self.device:
            self._bad("a cache", t, "a [blocks, ...] tensor")
        if t.is_contiguous():
            blocks, all_bytes = shape[0], t.nbytes
            if all_bytes > 0:
                run = all_bytes // blocks
                return _CACHE.pack(t.data_ptr(), blocks, run, 0, 0, 1, 1, run)
        if 0 in shape[1:]:
            self._bad("a cache", t, "a tensor whose pages hold something")
        size, strides = t.element_size(), t.stride()
        # the loops over a page, the inner ones first; those that follow one another in memory are one
        run, loops = 1, []
        for stride, n in sorted((stride, n) for stride, n in zip(strides[1:], shape[1:]) if n > 1):
            if not loops and stride == run:
                run *= n
            elif loops and stride == loops[-1][0] * loops[-1][1]:
                loops[-1][1] *= n
            else:
                loops.append([stride, n])
        ends = 1  # of the dimensions so far, the pages' among them
        for stride, n in sorted((stride, n) for stride, n in zip(strides, shape) if n > 1):
            if stride < ends:
                self._bad("a cache", t, "a tensor whose elements do not overlap")
            ends += stride * (n - 1)
        if len(loops) > 2:
            self._bad("a cache", t, "a tensor whose pages are at most two loops over runs of memory")
        (s0, n0), (s1, n1) = (loops[::-1] + [[0, 1], [0, 1]])[:2]
        return _CACHE.pack(t.data_ptr(), shape[0], strides[0] * size, s0 * size, s1 * size, n0, n1, run * size)

    def copy_pages(self, caches, copies: PageCopies, stream=None) -> None:
        """Copies page ``copies.source[i]`` to ``copies.target[i]`` in every one of ``caches`` (tensors [blocks, ...]: layers' keys, values,
        scales, means; or what ``page_caches`` made of them); pairs with a -1 are skipped. No target may be listed twice, or as a source."""
        if not isinstance(caches, PageCaches):
            caches = self.page_caches(caches)
        elif caches.device != self.device:
            raise ValueError(f"caches on device {caches.device} for a decoder on {self._dev}")
        n = copies.source.numel()
        self._call(self._copy, _COPY.pack(self._ints("source", copies.source, n), self._ints("target", copies.target, n), n, caches.address,
                                          len(caches.tensors), self._workspace_ptr), stream)
