"""The calls around the selection, for torch tensors: a paged cache's map, the
indexer's logits, and attention over the cache.

Argument marshalling only, like the rest of the binding: shapes, strides and
types are read from the tensors, checked, and handed to ``libtopk.so``.
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


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class PagedDecoder:
    """The paged calls on one device, with their workspace.

    Calls that may overlap on the GPU need separate PagedDecoders. ``stream`` is a torch
    stream (default: the current one); tensors that were made on another stream must be
    ready there, and outlive the call, as with any kernel. Outputs made here belong to it.
    """

    def __init__(self, device: int = 0):
        import torch

        self._torch = torch
        self.device = device
        self._dev = torch.device("cuda", device)
        self._lib = _sar._load()
        self._dtypes = {torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}
        self.nbytes = _sar.topk_attention_workspace_size(device)
        if self.nbytes == 0:
            raise _sar.TopkError(_sar.TOPK_ERR_CUDA, "topk_attention_workspace_size")
        with torch.cuda.device(device):
            self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=self._dev)
            self.reset()

    def reset(self, stream=None) -> None:
        """Clears the status word (stream-ordered)."""
        rc = _sar.topk_workspace_init(self.workspace, _sar.TOPK_PAGED_WORKSPACE_BYTES, stream)
        if rc != _sar.TOPK_OK:
            raise _sar.TopkError(rc, "topk_workspace_init")

    def status(self, stream=None) -> int:
        """The sticky TOPK_DEV_* bits; synchronises the stream."""
        rc, word = _sar.topk_get_status(self.workspace, stream)
        if rc != _sar.TOPK_OK:
            raise _sar.TopkError(rc, "topk_get_status")
        return word

    def _on(self, t, what: str, dtype, dims: int):
        _need(t.dtype == dtype and t.dim() == dims, f"{what} must be a {dims}-dimensional {dtype} tensor")
        _need(t.device == self._dev, f"{what} must be on {self._dev}")
        return t.data_ptr()

    def _ints(self, t, what: str, n=None):
        p = self._on(t, what, self._torch.int32, 1)
        _need(t.is_contiguous() and (n is None or t.numel() == n), f"{what} must be contiguous" + ("" if n is None else f" with {n} entries"))
        return p

    def _empty(self, shape, dtype, stream):
        torch = self._torch
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self._dev)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self._dev)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self._dev)

    def _call(self, name: str, args: bytes, stream) -> None:
        torch = self._torch
        if stream is None:
            stream = torch.cuda.current_stream(self._dev)
        if not isinstance(stream, int):
            stream = stream.cuda_stream
        if torch.cuda.current_device() == self.device:
            rc = getattr(self._lib, name)(args, stream)
        else:
            with torch.cuda.device(self.device):
                rc = getattr(self._lib, name)(args, stream)
        if rc != _sar.TOPK_OK:
            raise _sar.TopkError(rc, name)

    def kv_map(self, context_lens, new_lens, block_table, free_blocks, taken, block_size: int, max_tokens: int,
               taken_out=None, out: KvMap | None = None, stream=None) -> KvMap:
        """Gives the requests' new tokens their places: enters the blocks taken from ``free_blocks`` in
        ``block_table`` (int32 [requests, columns], in place), advances ``taken`` (int32 [1]; into
        ``taken_out`` if that is given) and lists slot, length and request of every new token."""
        torch = self._torch
        n = context_lens.numel()
        context, new = self._ints(context_lens, "context_lens"), self._ints(new_lens, "new_lens", n)
        table = self._on(block_table, "block_table", torch.int32, 2)
        _need(block_table.shape[0] == n and block_table.stride(1) == 1, "block_table must hold one contiguous row per request")
        if out is None:
            out = KvMap(self._empty(max_tokens, torch.int64, stream), self._empty(max_tokens, torch.int32, stream),
                        self._empty(max_tokens, torch.int32, stream), self._empty(n + 1, torch.int32, stream))
        slots = self._on(out.slots, "out.slots", torch.int64, 1)
        _need(out.slots.is_contiguous() and out.slots.numel() == max_tokens, "out.slots must be contiguous with max_tokens entries")
        taken_ptr = self._ints(taken, "taken", 1)
        self._call("topk_kv_map", _MAP.pack(
            context, new, n, block_size, table, block_table.stride(0) if n > 1 else max(block_table.stride(0), block_table.shape[1]), block_table.shape[1],
            self._ints(free_blocks, "free_blocks"), free_blocks.numel(), taken_ptr,
            taken_ptr if taken_out is None else self._ints(taken_out, "taken_out", 1), slots,
            self._ints(out.row_lens, "out.row_lens", max_tokens), self._ints(out.row_request, "out.row_request", max_tokens),
            self._ints(out.token_start, "out.token_start", n + 1), max_tokens, self.workspace.data_ptr()), stream)
        return out

    def _rows(self, rows: int, lengths, block_table, num_blocks: int, block_size: int, next_n, row_request):
        torch = self._torch
        _need(lengths.dtype == torch.int32 and lengths.dim() in (1, 2) and lengths.is_contiguous() and lengths.device == self._dev,
              f"lengths must be a contiguous int32 tensor with 1 or 2 dimensions on {self._dev}")
        _need(lengths.numel() == rows, "lengths must hold one length per row")
        if next_n is None:
            next_n = lengths.shape[1] if lengths.dim() == 2 else 1
        table = self._on(block_table, "block_table", torch.int32, 2)
        requests, columns = block_table.shape
        _need(block_table.stride(1) == 1 or columns == 1, "block_table's rows must be contiguous")
        return (rows, next_n, block_size, requests, num_blocks, lengths.data_ptr(),
                None if row_request is None else self._ints(row_request, "row_request", rows), table,
                max(block_table.stride(0), columns) if requests < 2 else block_table.stride(0), columns)

    def _vectors(self, t, what: str, dtype, dims: int):
        p = self._on(t, what, dtype, dims)
        _need(t.stride(-1) == 1 or t.shape[-1] == 1, f"{what}'s last dimension must be contiguous")
        return p

    def index_logits(self, q, weights, keys, block_table, lengths, key_scales=None, next_n: int | None = None,
                     row_request=None, max_len: int | None = None, out=None, stream=None):
        """Scores of every cached token for every row: q [rows, heads, dim], weights fp32 [rows, heads],
        keys [blocks, block_size, dim] (fp16, bf16 or fp8 e4m3, as q), key_scales fp32 [blocks, block_size].
        Writes logits fp32 [rows, max_len] up to each row's length and leaves the rest of ``out`` as it is
        (what a new tensor holds there is undefined; the selection never uses it)."""
        torch = self._torch
        rows, heads, dim = q.shape
        _need(q.dtype in self._dtypes, f"q has an unsupported type {q.dtype}")
        qp, kp = self._vectors(q, "q", q.dtype, 3), self._vectors(keys, "keys", q.dtype, 3)
        wp = self._on(weights, "weights", torch.float32, 2)
        _need(weights.shape == (rows, heads) and (weights.stride(1) == 1 or heads == 1), "weights must be [rows, heads] with contiguous rows")
        _need(keys.shape[2] == dim, "q and keys must have the same last dimension")
        sp, s0, s1 = None, 0, 0
        if key_scales is not None:
            sp = self._on(key_scales, "key_scales", torch.float32, 2)
            _need(key_scales.shape == keys.shape[:2], "key_scales must be [blocks, block_size]")
            s0, s1 = key_scales.stride()
        rows_args = self._rows(rows, lengths, block_table, keys.shape[0], keys.shape[1], next_n, row_request)
        if out is None:
            out = self._empty((rows, block_table.shape[1] * keys.shape[1] if max_len is None else max_len), torch.float32, stream)
        op = self._on(out, "out", torch.float32, 2)
        _need(out.shape[0] == rows and (out.stride(1) == 1 or out.shape[1] == 1), "out must hold one contiguous row per row of q")
        _need(max_len is None or max_len <= out.shape[1], "max_len must not exceed out's columns")
        self._call("topk_index_logits", _LOGITS.pack(
            *(x or 0 for x in rows_args), self._dtypes[q.dtype], heads, dim, qp, q.stride(0), q.stride(1), wp, weights.stride(0), kp, keys.stride(0), keys.stride(1),
            sp or 0, s0, s1, op, out.stride(0), out.shape[1] if max_len is None else max_len, self.workspace.data_ptr()), stream)
        return out

    def attention(self, q, k_cache, block_table, lengths, v_cache=None, v_dim: int | None = None, indices=None,
                  scale: float | None = None, next_n: int | None = None, row_request=None, out=None, lse=None,
                  return_lse: bool = False, stream=None):
        """Attention of q [rows, heads, dk] over a paged cache [blocks, block_size, kv_heads, dk] (or without
        the heads' dimension), over every token below each row's length or over ``indices``
        (int32 [rows, n], as the selection writes them). ``v_cache`` None: a token's value is the first
        ``v_dim`` elements of its key (latent attention). Returns out, or (out, lse)."""
        torch = self._torch
        if k_cache.dim() == 3:
            k_cache = k_cache.unsqueeze(2)
        if v_cache is not None and v_cache.dim() == 3:
            v_cache = v_cache.unsqueeze(2)
        rows, heads, dk = q.shape
        _need(q.dtype in self._dtypes, f"q has an unsupported type {q.dtype}")
        qp, kp = self._vectors(q, "q", q.dtype, 3), self._vectors(k_cache, "k_cache", q.dtype, 4)
        blocks, block_size, kv_heads, _ = k_cache.shape
        _need(k_cache.shape[3] == dk, "q and k_cache must have the same last dimension")
        vp, vs = 0, (0, 0, 0, 0)
        if v_cache is not None:
            vp, vs = self._vectors(v_cache, "v_cache", q.dtype, 4), v_cache.stride()
            _need(v_cache.shape[:3] == k_cache.shape[:3] and v_dim in (None, v_cache.shape[3]), "v_cache must have k_cache's blocks and heads, and v_dim values")
            v_dim = v_cache.shape[3]
        _need(v_dim is not None, "v_dim must be given where there is no v_cache")
        ip, i0, topk = 0, 0, 0
        if indices is not None:
            ip = self._on(indices, "indices", torch.int32, 2)
            _need(indices.shape[0] == rows and (indices.stride(1) == 1 or indices.shape[1] == 1), "indices must hold one contiguous row per row of q")
            i0, topk = indices.stride(0), indices.shape[1]
        rows_args = self._rows(rows, lengths, block_table, blocks, block_size, next_n, row_request)
        if out is None:
            out = self._empty((rows, heads, v_dim), q.dtype, stream)
        op = self._vectors(out, "out", q.dtype, 3)
        _need(out.shape == (rows, heads, v_dim), "out must be [rows, heads, v_dim]")
        if lse is None and return_lse:
            lse = self._empty((rows, heads), torch.float32, stream)
        lp = 0
        if lse is not None:
            lp = self._on(lse, "lse", torch.float32, 2)
            _need(lse.shape == (rows, heads) and lse.is_contiguous(), "lse must be a contiguous [rows, heads] tensor")
        ks = k_cache.stride()
        self._call("topk_paged_attention", _ATTENTION.pack(
            *(x or 0 for x in rows_args), self._dtypes[q.dtype], heads, kv_heads, dk, v_dim, dk ** -0.5 if scale is None else scale, qp, q.stride(0), q.stride(1),
            kp, ks[0], ks[1], ks[2], vp, vs[0], vs[1], vs[2], ip, i0, topk, op, out.stride(0), out.stride(1), lp, self.workspace.data_ptr(), self.nbytes), stream)
        return (out, lse) if return_lse else out
