"""Samples of prompts over a paged cache, with this library's calls only:

    map        which pages the prompts' and the samples' new tokens go to       PagedDecoder.kv_map
    (write)    their keys and values into the pages                             torch indexing
    means      the mean keys of the pages written to                            PagedDecoder.block_means
    fork       samples share their prompt's whole pages and copy the last one   PagedDecoder.fork_pages, copy_pages
    attend     a dense layer: the prompt is read once for all of its samples    PagedDecoder.shared_attention
               a sparse layer: blocks chosen by their mean keys                 PagedDecoder.block_scores, Selector, block_attention
    drop       samples that are not followed, and others forked anew            PagedDecoder.free_pages, fork_pages
    compact    the pool's highest pages moved to the lowest numbers             PagedDecoder.compact_pages, copy_pages

Run `python examples/shared_prompts.py`. Every step's attention is checked against the definition in 64 bits over tokens kept beside
the cache.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_row_gb300 as sar  # noqa: E402


class Pool:
    """One layer's pages and the tables over them; rows of the table are requests. What a model would compute is drawn instead."""

    def __init__(self, requests: int, columns: int, pages: int, block: int, kv_heads: int, dim: int, seed: int):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.block, self.kv_heads, self.dim = block, kv_heads, dim
        ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.k, self.v = (torch.full((pages, block, kv_heads, dim), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.means = torch.zeros((pages, kv_heads, dim), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((requests, columns), -1, dtype=torch.int32, device="cuda")
        self.free, self.taken, self.shares = torch.randperm(pages, generator=self.g, device="cuda").int(), ints(1), ints(pages)
        self.context = ints(requests)
        self.decoder, self.selector = sar.PagedDecoder(torch.cuda.current_device()), sar.Selector(torch.cuda.current_device())
        self.caches = self.decoder.page_caches([self.k, self.v, self.means])
        self.told = [torch.zeros(2, 0, kv_heads, dim) for _ in range(requests)]  # on the host, for the checks alone

    def draw(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.bfloat16)

    def grow(self, new):
        """Brings new[r] tokens to each request."""
        lens, total = torch.tensor(new, dtype=torch.int32, device="cuda"), sum(new)
        m = self.decoder.kv_map(self.context, lens, self.table, self.free, self.taken, self.block, total)
        fresh = self.draw(2, total, self.kv_heads, self.dim)
        for cache, x in ((self.k, fresh[0]), (self.v, fresh[1])):
            cache.view(-1, self.kv_heads, self.dim)[m.slots] = x
        self.decoder.block_means(self.k, self.table, self.context, lens, self.means)
        self.context += lens
        for r, piece in enumerate(fresh.float().cpu().split(new, 1)):
            self.told[r] = torch.cat([self.told[r], piece], 1)

    def drop(self, requests):
        self.decoder.free_pages(torch.tensor(requests, dtype=torch.int32, device="cuda"), self.table, self.shares, self.free, self.taken)
        self.context[requests] = 0
        for r in requests:
            self.told[r] = self.told[r][:, :0]

    def fork(self, parents, children):
        """The children become what their parents are."""
        a, b = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (parents, children))
        copies = self.decoder.fork_pages(a, b, self.context[a.long()], self.table, self.shares, self.free, self.taken, self.block)
        self.decoder.copy_pages(self.caches, copies)
        self.context[children] = self.context[parents]
        for x, y in zip(parents, children):
            self.told[y] = self.told[x].clone()

    def compact(self, most: int):
        moves = self.decoder.compact_pages(self.table, self.shares, self.free, self.taken, most)
        self.decoder.copy_pages(self.caches, moves)


def dense(pool: Pool, q, prefix_of, prefix_lens, prefix_rows, longest: int):
    """Attention over everything, prompts read once. The prompts' table is as wide as the longest of them: the call goes by that."""
    prefixes = pool.table[prefix_rows, :max(longest // pool.block, 1)]
    return pool.decoder.shared_attention(q, pool.k, pool.table, pool.context, prefix_of, prefix_lens, prefixes, v_cache=pool.v)


def sparse(pool: Pool, q, topk: int):
    """Attention over the best blocks, the first and the last ones among them."""
    scores, lens = pool.decoder.block_scores(q, pool.means, pool.table, pool.context, pool.block, sink_blocks=1, recent_blocks=1)
    chosen = pool.selector(scores.flatten(0, 1), lens.flatten(), topk).view(*lens.shape, topk)
    return pool.decoder.block_attention(q, pool.k, pool.table, pool.context, chosen, v_cache=pool.v), chosen


def check(pool: Pool, q, out, chosen=None) -> float:
    """The largest distance of `out` from attention in 64 bits, on the host."""
    worst, group = 0.0, q.shape[1] // pool.kv_heads
    q, out, chosen = q.cpu().double(), out.cpu().double(), None if chosen is None else chosen.cpu()
    for r, (k, v) in enumerate(pool.told):
        for h in range(pool.kv_heads):
            t = torch.arange(len(k))
            if chosen is not None:
                t = t[(t[:, None] // pool.block == chosen[r, h]).any(1)]
            if len(t) == 0:
                continue
            s = q[r, h * group:(h + 1) * group] @ k[t, h].double().T * pool.dim ** -0.5
            want = torch.softmax(s, -1) @ v[t, h].double()
            worst = max(worst, float((out[r, h * group:(h + 1) * group] - want).abs().max()))
    return worst


def run(prompts: int = 2, samples: int = 4, tokens: int = 300, steps: int = 3, block: int = 16, heads: int = 8, kv_heads: int = 2, dim: int = 64, topk: int = 6, seed: int = 0) -> float:
    """Prompts, their samples, decode steps, samples dropped and drawn anew, the pool compacted; the largest distance from 64 bits."""
    requests = prompts * (1 + samples)
    pool = Pool(requests, -(-(tokens + 4 * steps) // block) + 1, 3 * requests * (tokens // block + 3), block, kv_heads, dim, seed)
    lengths = [tokens - 7 * i for i in range(prompts)]
    pool.grow(lengths + [0] * (requests - prompts))
    children = list(range(prompts, requests))  # the samples of a prompt lie side by side
    pool.fork([(c - prompts) // samples for c in children], children)
    prefix_of = torch.tensor([-1] * prompts + [(c - prompts) // samples for c in children], dtype=torch.int32, device="cuda")
    prefix_lens, prefix_rows = torch.tensor(lengths, dtype=torch.int32, device="cuda"), list(range(prompts))
    worst = 0.0
    for step in range(2 * steps):
        if step == steps:  # the last sample of each prompt starts anew from the first one
            last = [prompts + i * samples + samples - 1 for i in range(prompts)]
            pool.drop(last)
            pool.fork([prompts + i * samples for i in range(prompts)], last)
            pool.compact(1000)
        pool.grow([0] * prompts + [1 + (r + step) % 2 for r in range(requests - prompts)])
        q = pool.draw(requests, heads, dim)
        worst = max(worst, check(pool, q, dense(pool, q, prefix_of, prefix_lens, prefix_rows, max(lengths))))
        out, chosen = sparse(pool, q, topk)
        worst = max(worst, check(pool, q, out, chosen))
    pool.drop(list(range(requests)))
    assert int(pool.taken) == 0 and not pool.shares.any(), "pages were lost"
    for what, status in (("decoder", pool.decoder.status()), ("selector", pool.selector.status())):
        assert status == 0, f"{what}: device status {status:#x}"
    return worst


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", type=int, default=2)
    ap.add_argument("--samples", type=int, default=32)
    ap.add_argument("--tokens", type=int, default=4000)
    a = ap.parse_args()
    far = run(a.prompts, a.samples, a.tokens, heads=32, kv_heads=8, dim=128, block=64, topk=16)
    print(f"{a.prompts} prompts of about {a.tokens} tokens, {a.samples} samples each: largest distance from 64 bits {far:.4f}")


if __name__ == "__main__":
    main()
