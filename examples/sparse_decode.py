"""Sparse-attention decoding over a paged cache, with this library's calls only:

    map        which pages the new tokens go to, and what each of them sees   PagedDecoder.kv_map
    (write)    the new tokens' latent vectors and indexer keys into the pages  torch indexing
    score      every cached token, by the indexer                             PagedDecoder.index_logits
    select     the best TopK of them                                          Selector
    attend     latent attention over the selection                            PagedDecoder.attention

Run `python examples/sparse_decode.py`: a prompt for each request, then decode steps. Every step is checked against plain
attention in 64 bits over the tokens that were selected, and the selection against a sort of the logits.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_row_gb300 as sar  # noqa: E402


class Layer:
    """One layer's caches and fixed random projections; what a model would compute is drawn instead."""

    def __init__(self, requests: int, tokens: int, block: int, heads: int, index_heads: int, seed: int):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.block, self.heads, self.index_heads = block, heads, index_heads
        columns = -(-tokens // block)
        self.blocks = requests * columns
        self.latent = torch.full((self.blocks, block, 1, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.keys = torch.full((self.blocks, block, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((requests, columns), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.blocks, generator=self.g, device="cuda", dtype=torch.int32)
        self.taken = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.context = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def draw(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.bfloat16)


def step(layer: Layer, decoder: sar.PagedDecoder, selector: sar.Selector, new: torch.Tensor, rows: int, topk: int):
    """Brings `new` tokens (int32 [requests], `rows` in all) through the layer; returns what the calls made."""
    m = decoder.kv_map(layer.context, new, layer.table, layer.free, layer.taken, layer.block, rows)
    layer.latent.view(-1, 576)[m.slots] = layer.draw(rows, 576)
    layer.keys.view(-1, 128)[m.slots] = layer.draw(rows, 128)
    layer.context += new
    q_index = layer.draw(rows, layer.index_heads, 128)
    weights = torch.randn((rows, layer.index_heads), generator=layer.g, device="cuda") / layer.index_heads
    logits = decoder.index_logits(q_index, weights, layer.keys, layer.table, m.row_lens, row_request=m.row_request)
    picked = selector(logits, m.row_lens, topk)
    q = layer.draw(rows, layer.heads, 576)
    out, lse = decoder.attention(q, layer.latent, layer.table, m.row_lens, v_dim=512, indices=picked, row_request=m.row_request, return_lse=True)
    return m, q_index, weights, logits, picked, q, out, lse


def check(layer: Layer, rows, m, q_index, weights, logits, picked, q, out, lse) -> float:
    """The largest distance of `out` from attention in 64 bits over a selection made by a sort."""
    worst = 0.0
    for r in rows:
        n, request = int(m.row_lens[r]), int(m.row_request[r])
        pos = torch.arange(n, device="cuda")
        slot = layer.table[request, pos // layer.block].long() * layer.block + pos % layer.block
        score = (weights[r].double()[:, None] * torch.relu(q_index[r].double() @ layer.keys.view(-1, 128)[slot].double().T)).sum(0)
        assert (logits[r, :n].double() - score).abs().max() < 1e-4, f"row {r}: logits"
        best = torch.sort(logits[r, :n], descending=True, stable=True).indices[:picked.shape[1]]
        got = picked[r][picked[r] >= 0]
        assert torch.equal(best.sort().values, got.long().sort().values), f"row {r}: selection"
        kv = layer.latent.view(-1, 576)[slot[best]].double()
        s = q[r].double() @ kv.T * 576 ** -0.5
        want = torch.softmax(s, -1) @ kv[:, :512]
        worst = max(worst, float((out[r].double() - want).abs().max()))
        assert (lse[r].double() - torch.logsumexp(s, -1)).abs().max() < 1e-3, f"row {r}: lse"
    return worst


def run(requests: int = 6, prompt: int = 700, steps: int = 4, topk: int = 512, block: int = 64, heads: int = 16, seed: int = 0) -> float:
    layer = Layer(requests, prompt + 2 * steps, block, heads, 32, seed)
    decoder, selector = sar.PagedDecoder(torch.cuda.current_device()), sar.Selector(torch.cuda.current_device())
    lengths = [1 + (prompt - 1) * (r + 1) // requests for r in range(requests)]
    worst = 0.0
    for s in range(steps + 1):
        # the prompts first, then one or two tokens (a drafted one) for each request
        count = lengths if s == 0 else [1 + (r + s) % 2 for r in range(requests)]
        rows = sum(count)
        made = step(layer, decoder, selector, torch.tensor(count, dtype=torch.int32, device="cuda"), rows, topk)
        some = range(0, rows, max(1, rows // 16))
        worst = max(worst, check(layer, some, *made))
    for what, status in (("decoder", decoder.status()), ("selector", selector.status())):
        assert status == 0, f"{what}: device status {status:#x}"
    return worst


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=8192)
    ap.add_argument("--topk", type=int, default=2048)
    ap.add_argument("--heads", type=int, default=16)
    a = ap.parse_args()
    print(f"checked against 64 bits: largest distance {run():.4f}")
    layer = Layer(a.requests, a.prompt + 64, 64, a.heads, 64, 1)
    decoder, selector = sar.PagedDecoder(torch.cuda.current_device()), sar.Selector(torch.cuda.current_device())
    fill = torch.full((a.requests,), a.prompt, dtype=torch.int32, device="cuda")
    m = decoder.kv_map(layer.context, fill, layer.table, layer.free, layer.taken, 64, a.requests * a.prompt)
    layer.latent.view(-1, 576)[m.slots] = layer.draw(a.requests * a.prompt, 576)
    layer.keys.view(-1, 128)[m.slots] = layer.draw(a.requests * a.prompt, 128)
    layer.context += fill
    one = torch.ones_like(fill)
    for _ in range(8):
        step(layer, decoder, selector, one, a.requests, a.topk)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(32):
        step(layer, decoder, selector, one, a.requests, a.topk)
    torch.cuda.synchronize()
    print(f"{a.requests} requests, about {a.prompt} tokens each, TopK {a.topk}, {a.heads} heads: {(time.perf_counter() - t) / 32 * 1e6:.0f} us a step, "
          "what stands for the model included")


if __name__ == "__main__":
    main()
