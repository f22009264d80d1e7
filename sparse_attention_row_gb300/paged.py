"""The calls around the selection, for torch tensors: a paged cache's map, the
indexer's logits, and attention over the cache.

Argument marshalling only, like the rest of the binding: shapes, strides and
types are read from the tensors, checked, and handed to ``libtopk.so``. A decode
step makes these calls back to back, so the checks are plain comparisons and the
arguments are packed in one go: a call with its outputs given is enqueued in 7 to 10 us of host time.
"""
from __future__ import annotations

import struct
from typing import NamedTuple

import sparse_attention_row_gb300 as _sar

# The argument structs of include/libtopk.h in order, with native sizes and alignment
# (tests/test_paged_cpu.py compares them with the header's).
_ROWS = "qiiqqPPPqq"
_MAP = struct.Struct("@PPqiPqqPqPPPPPPqP")
_LOGITS = struct.Struct("@" + _ROWS + "iiiPqqPqPqqPqqPqqP")
_ATTENTION = struct.Struct("@" + _ROWS + "iiiiifPqqPqqqPqqqPqiPqqPPN")


class KvMap(NamedTuple):
    """What ``PagedDecoder.kv_map`` lists for the new tokens of a step, packed request after request."""
    slots: "torch.Tensor"        # int64 [max_tokens], flat cache positions, -1 where there is none  # noqa: F821
    row_lens: "torch.Tensor"     # int32 [max_tokens], position + 1: the rows' lengths  # noqa: F821
    row_request: "torch.Tensor"  # int32 [max_tokens], -1 past the last token  # noqa: F821
    token_start: "torch.Tensor"  # int32 [requests + 1]  # noqa: F821


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
        self._f32, self._i32, self._i64 = torch.float32, torch.int32, torch.int64
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
        return p, s0, s1, s2, shape[:3], shape[3]

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
        requests = len(block_table)
        table, stride, columns = self._matrix("block_table", block_table, self._i32, requests)
        return (rows, next_n, block_size, requests, num_blocks, lengths.data_ptr(),
                0 if row_request is None else self._ints("row_request", row_request, rows), table,
                stride if requests > 1 or stride >= columns else columns, columns)

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

    def attention(self, q, k_cache, block_table, lengths, v_cache=None, v_dim: int | None = None, indices=None,
                  scale: float | None = None, next_n: int | None = None, row_request=None, out=None, lse=None,
                  return_lse: bool = False, stream=None):
        """Attention of q [rows, heads, dk] over a paged cache [blocks, block_size, kv_heads, dk] (or without
        the heads' dimension), over every token below each row's length or over ``indices``
        (int32 [rows, n], as the selection writes them). ``v_cache`` None: a token's value is the first
        ``v_dim`` elements of its key (latent attention). Returns out, or (out, lse)."""
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
        self._call(self._attention, _ATTENTION.pack(
            *rows_args, kind, heads, kv_heads, dk, v_dim, dk ** -0.5 if scale is None else scale, qp, q0, q1,
            kp, k0, k1, k2, vp, v0, v1, v2, ip, i0, topk, op, o0, o1, lp, self._workspace_ptr, self.nbytes), stream)
        return (out, lse) if return_lse else out
