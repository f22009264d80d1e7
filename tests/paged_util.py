"""Inputs and 64-bit definitions for the tests of the paged calls."""
from __future__ import annotations

import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a unit in the last place, relative
ACC = 2.0 ** -22  # relative step of a fp32 sum, twice the unit for products that are summed in another order


def block_table(g, lengths, block, spare=2, columns=None):
    """A table whose pages come in random order, -1 past each request's last, and the number of blocks."""
    used = [-(-int(n) // block) for n in lengths]
    order = torch.randperm(sum(used) + spare, generator=g).tolist()
    columns = max(used + [1]) if columns is None else columns
    rows, at = [], 0
    for u in used:
        rows.append(order[at:at + u] + [-1] * (columns - u))
        at += u
    return torch.tensor(rows, dtype=torch.int32).reshape(len(used), columns), sum(used) + spare


def poisoned(cache, table, lengths, block):
    """The cache with NaN everywhere that no request's token lies."""
    keep = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for r, n in enumerate(lengths):
        t = torch.arange(int(n))
        keep[table[r, t // block].long(), t % block] = True
    bad = torch.full_like(cache, math.nan, dtype=torch.float32).to(cache.dtype)
    return torch.where(keep.reshape(keep.shape + (1,) * (cache.dim() - 2)), cache, bad) if cache.dtype != torch.float8_e4m3fn else \
        torch.where(keep.reshape(keep.shape + (1,) * (cache.dim() - 2)), cache.view(torch.uint8), bad.view(torch.uint8)).view(cache.dtype)


def tokens(table, request, positions, block):
    return table[request, positions // block].long(), positions % block


def logits64(q, w, keys, scales, table, lengths, requests, block, max_len):
    """(logits, bound of their error) in 64 bits; nan past each row's length."""
    rows = q.shape[0]
    out = torch.full((rows, max_len), math.nan, dtype=torch.float64)
    tol = out.clone()
    for r in range(rows):
        pos = torch.arange(min(int(lengths[r]), max_len))
        b, o = tokens(table, requests[r], pos, block)
        k, qq, ww = keys.to(torch.float32)[b, o].double(), q.to(torch.float32)[r].double(), w[r].double()
        s = scales[b, o].double() if scales is not None else torch.ones(len(pos), dtype=torch.float64)
        out[r, :len(pos)] = (ww[:, None] * (qq @ k.T).clamp(min=0)).sum(0) * s
        size = (ww.abs()[:, None] * (qq.abs() @ k.abs().T)).sum(0) * s
        tol[r, :len(pos)] = size * (q.shape[1] + q.shape[2] + 4) * ACC + 1e-30
    return out, tol


def attention64(q, k, v, dv, table, lengths, requests, block, scale, indices=None):
    """(out, lse, bound of out's error without its own rounding, bound of lse's) in 64 bits, and sum of p |v|."""
    rows, heads, dk = q.shape
    kv_heads = k.shape[2]
    group = heads // kv_heads
    out = torch.zeros(rows, heads, dv, dtype=torch.float64)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    u = U[q.dtype]
    for r in range(rows):
        n = int(lengths[r])
        pos = torch.arange(n) if indices is None else indices[r].long()
        pos = pos[(pos >= 0) & (pos < n)]
        if len(pos) == 0:
            continue
        b, o = tokens(table, requests[r], pos, block)
        for h in range(kv_heads):
            kk = k[b, o, h].double()
            vv = kk[:, :dv] if v is None else v[b, o, h].double()
            sl = slice(h * group, (h + 1) * group)
            qq = q[r, sl].double()
            s = qq @ kk.T * scale
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = torch.exp(s - m)
            total = p.sum(-1, keepdim=True)
            seen = total > 0
            out[r, sl] = torch.where(seen, p @ vv / total.clamp(min=1e-300), 0.0)
            lse[r, sl] = torch.where(seen, m + total.log(), -math.inf)[:, 0]
            # a score's error, then the exponential's (two units of fp32 and its argument's rounding)
            fin = torch.where(kk.isfinite(), kk, 0.0)
            e = ((qq.abs() @ fin.abs().T) * scale).amax(-1, keepdim=True) * (dk + 4) * ACC + 2.0 ** -20
            mean = torch.where(seen, p @ vv.abs() / total.clamp(min=1e-300), 0.0)
            tol[r, sl] = mean * (u + 2 * e + len(pos) * ACC)
            ltol[r, sl] = (e + (len(pos) + 8) ** 0.5 * ACC + lse[r, sl].abs()[:, None].clamp(max=1e30) * 2.0 ** -22)[:, 0]
    return out, lse, tol, ltol


def check_attention(got, got_lse, want, dtype):
    out, lse, tol, ltol = want
    got, got_lse = got.cpu().double(), got_lse.cpu().double()
    room = tol + out.abs() * U[dtype] * (1 + 2.0 ** -6) + (2.0 ** -24 if dtype == torch.float16 else 1e-38)
    far = (got - out).abs()
    assert torch.isfinite(got).all()
    assert (far <= room).all(), f"out is {float((far / room).max()):.2f} of its bound off at {(far / room).argmax()}"
    empty = lse == -math.inf
    assert (got_lse[empty] == -math.inf).all() and (got[empty] == 0).all()
    lfar = (got_lse[~empty] - lse[~empty]).abs()
    assert (lfar <= ltol[~empty]).all(), f"lse is {float((lfar / ltol[~empty]).max()):.2f} of its bound off"
