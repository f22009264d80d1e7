"""Further forms of the calls for blocks, shared prefixes and pages: streams, graphs, plain launch order, steps back to back."""
import os
import subprocess
import sys

import pytest
import torch

import sparse_attention_row_gb300 as sar
from tests import paged_util as pu
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("switch", ["1", "2"])
def test_example_with_and_without_dependent_launch(switch):
    code = ("import importlib.util as u; s = u.spec_from_file_location('e', 'examples/shared_prompts.py'); m = u.module_from_spec(s); "
            "s.loader.exec_module(m); assert m.run(prompts=2, samples=5, tokens=333, heads=16, kv_heads=4, dim=64) < 3 * 2.0 ** -8 * 5")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, env=dict(os.environ, LIBTOPK_DEPENDENT_LAUNCH=switch), timeout=300)


class Step:
    """A step over blocks and one over a shared prefix, with all its tensors made beforehand."""

    def __init__(self, seed, rows=24, block=16, kv=2, heads=8, dim=64, prefix=200, topk=4):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.block, self.topk, self.rows, self.kv = block, topk, rows, kv
        full, columns = prefix // block, (prefix + 100) // block + 1
        pages = full + rows * (columns - full)
        r = lambda *s: torch.randn(s, generator=self.g, device="cuda").bfloat16()  # noqa: E731
        self.k, self.v, self.q = r(pages, block, kv, dim), r(pages, block, kv, dim), r(rows, heads, dim)
        self.table = torch.empty(rows, columns, dtype=torch.int32, device="cuda")
        self.table[:, :full] = torch.arange(full, device="cuda")
        self.table[:, full:] = torch.arange(full, pages, device="cuda").view(rows, -1)
        self.lens = ints([prefix + (17 * i) % 100 for i in range(rows)])
        self.zero, self.of, self.plen = ints([0] * rows), ints([0] * rows), ints([prefix])
        # wide enough that the prefix is shared even by so few rows
        self.prefix = torch.full((1, 300000), -1, dtype=torch.int32, device="cuda")
        self.prefix[0, :full] = torch.arange(full, device="cuda")
        self.means = torch.zeros(pages, kv, dim, device="cuda").bfloat16()
        self.decoder, self.selector = sar.PagedDecoder(0), sar.Selector(0)

    def run(self, stream=None):
        d = self.decoder
        d.block_means(self.k, self.table, self.zero, self.lens, self.means, stream=stream)
        scores, lens = d.block_scores(self.q, self.means, self.table, self.lens, self.block, sink_blocks=1, recent_blocks=1, stream=stream)
        chosen = self.selector(scores.flatten(0, 1), lens.flatten(), self.topk, stream=stream).view(self.rows, self.kv, self.topk)
        out = d.block_attention(self.q, self.k, self.table, self.lens, chosen, v_cache=self.v, return_lse=True, stream=stream)
        both = d.shared_attention(self.q, self.k, self.table, self.lens, self.of, self.plen, self.prefix, v_cache=self.v, return_lse=True, stream=stream)
        return [lens, *out, *both]  # the order of the chosen blocks, and what stands behind a row's scores, are unspecified

    def check(self, got):
        k, v, q, table, lens = self.k.cpu(), self.v.cpu(), self.q.cpu(), self.table.cpu(), self.lens.tolist()
        want = pu.attention64(q, k, v, v.shape[-1], table, lens, list(range(self.rows)), self.block, q.shape[-1] ** -0.5)
        pu.check_attention(got[3], got[4], (want[0], want[1], want[2] * 2.1, want[3] + 1e-5), torch.bfloat16)


def near(a, b):
    # chosen blocks may stand in another order: sums in another order, and probabilities' roundings by another first maximum
    assert torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[3:], b[3:]))
    assert (a[1].float() - b[1].float()).abs().max() <= 4 * 2.0 ** -8 * 5 and (a[2] - b[2]).abs().max() < 1e-4


def test_two_decoders_on_two_streams_at_once():
    steps = [Step(1), Step(2, rows=33, kv=4, heads=16)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        s.check(w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [s.run(stream) for s, stream in zip(steps, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            near(g, w)
    assert all(s.decoder.status() == 0 for s in steps)


def test_steps_back_to_back_and_in_graphs_of_one_decoder():
    step = Step(3)
    want = step.run()
    many = [step.run() for _ in range(15)]  # nothing waits between them
    torch.cuda.synchronize()
    for got in many:
        near(got, want)
    graphs, made = [], []
    for _ in range(2):  # two graphs of the same decoder, replayed in turn on one stream
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            made.append(step.run())
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for got in made:
        near(got, want)
    # other lengths, keys and prefixes where they stand
    step.k.copy_(torch.randn(step.k.shape, generator=step.g, device="cuda"))
    step.lens.add_(ints([i % 5 for i in range(step.rows)]))
    step.plen.fill_(100)
    for graph in graphs:
        graph.replay()
    want = step.run()
    torch.cuda.synchronize()
    step.check(want)
    for got in made:
        near(got, want)
    assert step.decoder.status() == 0


def test_pages_in_a_graph():
    pages, block, d = 64, 4, sar.PagedDecoder(0)
    table = torch.full((6, 8), -1, dtype=torch.int32, device="cuda")
    free, taken, shares = torch.randperm(pages, device="cuda").int(), ints([0]), ints([0] * pages)
    cache = torch.randn(pages, block, 24, device="cuda")
    context, new = ints([0] * 6), ints([27, 14, 0, 0, 0, 0])
    m = d.kv_map(context, new, table, free, taken, block, 41)
    parents, children, kept = ints([0, 1, 0]), ints([2, 3, 4]), ints([27, 14, 9])
    state = [x.clone() for x in (table, shares, free, taken)]

    def turn():
        copies = d.fork_pages(parents, children, kept, table, shares, free, taken, block)
        d.copy_pages([cache], copies)
        forked = [table.clone(), shares.clone(), taken.clone(), cache[copies.target.long().clamp(min=0)], cache[copies.source.long().clamp(min=0)]]
        d.free_pages(children, table, shares, free, taken)
        return forked

    want = turn()
    assert int(want[2]) == int(state[3]) + 3 and torch.equal(want[3], want[4]) and want[1].sum() == 6 + 3 + 2
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = turn()
    for _ in range(10):  # every turn leaves what it found
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip((table, shares, free, taken), state))
    assert d.status() == 0 and (m.slots >= 0).all()


def test_caches_and_tensors_that_are_refused():
    d = sar.PagedDecoder(0)
    q, k = torch.zeros(2, 4, 64, device="cuda").half(), torch.zeros(4, 16, 2, 64, device="cuda").half()
    table, lens, means = ints([[0, 1], [2, 3]]), ints([5, 20]), torch.zeros(4, 2, 64, device="cuda").half()
    for wrong in (lambda: d.block_scores(q, means, table, lens, 16, out=torch.zeros(2, 3, 2, device="cuda")),
                  lambda: d.block_scores(q, means[..., :32], table, lens, 16), lambda: d.block_scores(q.float(), means, table, lens, 16),
                  lambda: d.block_means(k, table, lens, lens, means[:3]), lambda: d.block_means(k, table, lens.long(), lens, means),
                  lambda: d.block_attention(q, k, table, lens, ints([[0], [1], [0]]), v_cache=k), lambda: d.block_attention(q, k, table, lens, torch.zeros(2, 2, 1, device="cuda"), v_cache=k),
                  lambda: d.block_attention(q, k, table, lens, torch.zeros(2, 3, 1, device="cuda").int(), v_cache=k),
                  lambda: d.shared_attention(q, k, table, lens, ints([0]), ints([3]), table[:1], v_cache=k), lambda: d.shared_attention(q, k, table, lens, ints([0, 0]), ints([3, 4]), table[:1], v_cache=k),
                  lambda: d.free_pages(lens.long(), table, ints([0] * 4), ints([0]), ints([0])), lambda: d.fork_pages(lens, ints([0]), lens, table, ints([0] * 4), ints([0]), ints([0]), 16),
                  lambda: d.copy_pages([k.cpu()], sar.PageCopies(ints([0]), ints([1]))), lambda: d.copy_pages([k] * 257, sar.PageCopies(ints([0]), ints([1]))),
                  lambda: d.copy_pages([k], sar.PageCopies(ints([0]), ints([1, 2]))), lambda: d.compact_pages(table, ints([0] * 4), ints([0]), ints([0]), 3, table_out=table[:, :1])):
        with pytest.raises(ValueError):
            wrong()
    with pytest.raises(sar.TopkError):  # what the library itself refuses
        d.block_scores(q, means, table, lens, 0)
    assert d.status() == 0
