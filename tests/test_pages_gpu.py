"""Forking, freeing, compacting and copying pages, against the same done one entry at a time; and all calls in a run together."""
import math
import random

import pytest
import torch

import sparse_attention_row_gb300 as sar
from tests import paged_util as pu
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dec():
    require_cuda()
    return sar.PagedDecoder(0)


@pytest.fixture(autouse=True)
def _clear(request):
    yield
    if "dec" in request.fixturenames:
        request.getfixturevalue("dec").reset()


def ok(dec, allowed=0):
    assert dec.status() & ~allowed == 0, f"device status {dec.status():#x}"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """The definition, a page at a time."""

    def __init__(self, rows, columns, pages, block, rng):
        self.block, self.columns = block, columns
        self.table = [[-1] * columns for _ in range(rows)]
        self.shares, self.taken = [0] * pages, 0
        self.free = rng.sample(range(pages), pages)

    def grow(self, row, tokens):
        for c in range(-(-tokens // self.block)):
            if self.table[row][c] < 0:
                self.table[row][c] = self.free[self.taken]
                self.taken += 1

    def fork(self, parents, children, kept):
        pairs = []
        for a, b, n in zip(parents, children, kept):
            n = min(max(n, 0), self.columns * self.block)
            row, pair = [-1] * self.columns, (-1, -1)
            for c in range(n // self.block):
                row[c] = self.table[a][c]
                self.shares[row[c]] += 1
            if n % self.block:
                source = self.table[a][n // self.block]
                target = self.free[self.taken] if self.taken < len(self.free) else -1
                self.taken = min(self.taken + 1, len(self.free))
                row[n // self.block], pair = target, (source if target >= 0 else -1, target)
            self.table[b] = row
            pairs.append(pair)
        return [p[0] for p in pairs], [p[1] for p in pairs]

    def release(self, requests):
        back, held = [], {}
        for r in dict.fromkeys(requests):
            for page in self.table[r]:
                if page >= 0:
                    held[page] = held.get(page, 0) + 1
            back += [p for p in self.table[r] if p >= 0]
            self.table[r] = [-1] * self.columns
        for page, n in held.items():
            self.shares[page] -= n
        back = [p for p in dict.fromkeys(back) if self.shares[p] < 0]
        for p in back:
            self.shares[p] = 0
        self.taken -= len(back)
        self.free[self.taken:self.taken + len(back)] = back

    def compact(self, most):
        named = sorted({p for row in self.table for p in row if p >= 0}, reverse=True)
        holes = sorted(self.free[self.taken:])
        moves = [(a, b) for a, b in zip(named, holes) if b < a][:most]
        to = dict(moves)
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for a, b in moves:
            self.shares[b], self.shares[a] = self.shares[a], 0
        self.free[self.taken:] = sorted((set(holes) - {b for _, b in moves}) | {a for a, _ in moves})
        tail = [-1] * (most - len(moves))
        return [a for a, _ in moves] + tail, [b for _, b in moves] + tail

    def device(self):
        return ints(self.table), ints(self.shares), ints(self.free), ints([self.taken])

    def same(self, state):
        table, shares, free, taken = state
        assert table.tolist() == self.table, "table"
        assert shares.tolist() == self.shares, "shares"
        assert int(taken) == self.taken and free.tolist() == self.free, "free pages"


SHAPES = [(6, 4, 40, 16), (40, 9, 400, 8), (300, 33, 12000, 4), (64, 700, 50000, 1), (17, 1, 64, 33)]


@pytest.mark.parametrize("rows, columns, pages, block", SHAPES)
def test_forks_and_frees_and_compactions(dec, rows, columns, pages, block):
    rng = random.Random(rows)
    pool = Pool(rows, columns, pages, block, rng)
    used = set(range(rows // 2))
    for r in used:
        pool.grow(r, rng.randrange(columns * block + 1))
    state = pool.device()
    for step in range(12):
        idle = [r for r in range(rows) if r not in used]
        children = rng.sample(idle, rng.randrange(len(idle) + 1))
        parents = [rng.choice(sorted(used)) for _ in children] if used else []
        children = children[:len(parents)]
        lens = [rng.choice([0, 1, rng.randrange(columns * block + 1)]) for _ in children]
        # no more than the parent has pages for
        kept = [min(n, block * sum(p >= 0 for p in pool.table[a])) for n, a in zip(lens, parents)]
        if pages - pool.taken < len(kept):
            kept = [n // block * block for n in kept]
        copies = dec.fork_pages(ints(parents), ints(children), ints(kept), *state, block)
        assert (copies.source.tolist(), copies.target.tolist()) == pool.fork(parents, children, kept)
        pool.same(state)
        used |= set(children)
        gone = rng.sample(sorted(used), rng.randrange(len(used) + 1))
        listed = gone + gone[:2]  # some twice
        dec.free_pages(ints(listed), *state)
        pool.release(listed)
        pool.same(state)
        used -= set(gone)
        for r in rng.sample(sorted(used), len(used) // 3):
            if pages - pool.taken > columns:
                pool.grow(r, rng.randrange(columns * block + 1))
        state = pool.device()
        if step % 3 == 2:
            most = rng.choice([0, 1, 7, pages])
            new = [torch.full_like(x, -3) for x in state]
            copies = dec.compact_pages(*state, most, table_out=new[0], shares_out=new[1], free_out=new[2], taken_out=new[3])
            assert (copies.source.tolist(), copies.target.tolist()) == pool.compact(most)
            pool.same(new)
            again = dec.compact_pages(*state, most)  # the same in place
            pool.same(state)
            assert all(torch.equal(a, b) for a, b in zip(copies, again))
    ok(dec)


def test_shared_pages_go_back_once_in_the_order_of_their_first_places(dec):
    pool = Pool(5, 3, 12, 4, random.Random(1))
    pool.grow(0, 12)
    state = pool.device()
    for n in (12, 12, 8, 5):
        child = {12: 1, 8: 3, 5: 4}[n] if n != 12 or pool.table[1][0] < 0 else 2
        dec.fork_pages(ints([0]), ints([child]), ints([n]), *state, 4)
        pool.fork([0], [child], [n])
    pool.same(state)
    dec.free_pages(ints([3, 0]), *state)
    pool.release([3, 0])
    pool.same(state)
    dec.free_pages(ints([4, 2, 1]), *state)
    pool.release([4, 2, 1])
    pool.same(state)
    assert pool.taken == 0 and not any(pool.shares)
    ok(dec)


def test_many_requests_freed_at_once_the_same_every_time(dec):
    rng = random.Random(5)
    pool = Pool(1200, 20, 8000, 2, rng)
    for r in range(300):
        pool.grow(r, rng.randrange(41))
    parents, children = [rng.randrange(300) for _ in range(900)], list(range(300, 1200))
    kept = [2 * sum(p >= 0 for p in pool.table[a]) for a in parents]
    pool.fork(parents, children, kept)
    gone = rng.sample(range(1200), 1000)
    states = [pool.device() for _ in range(4)]
    pool.release(gone)
    for s in states:
        dec.free_pages(ints(gone), *s)
        pool.same(s)
    ok(dec)


def test_wide_tables_freed_in_several_rounds(dec):
    rng = random.Random(6)
    pool = Pool(400, 700, 60000, 1, rng)
    for r in range(100):
        pool.grow(r, rng.randrange(300, 500))
    parents = [rng.randrange(100) for _ in range(300)]
    kept = [rng.randrange(sum(p >= 0 for p in pool.table[a]) + 1) for a in parents]
    state = pool.device()
    dec.fork_pages(ints(parents), ints(list(range(100, 400))), ints(kept), *state, 1)
    pool.fork(parents, list(range(100, 400)), kept)
    pool.same(state)
    gone = rng.sample(range(400), 380)
    gone.insert(200, gone[3])
    dec.free_pages(ints(gone), *state)
    pool.release(gone)
    pool.same(state)
    dec.compact_pages(*state, 100000)
    pool.compact(100000)
    pool.same(state)
    ok(dec)


def test_fork_limits(dec):
    # no free page left; rows outside the table; a parent without the page; more tokens than the table is wide
    table = ints([[4, 5, 6], [7, -1, 90], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1], [9, 9, 9]])
    shares, free, taken = ints([0] * 12), ints([0, 1, 2]), ints([2])
    copies = dec.fork_pages(ints([0, 0, 9, 1, 0]), ints([2, 3, 4, 4, 5]), ints([5, 6, 4, 7, 100]), table, shares, free, taken, 4)
    assert copies.source.tolist() == [5, -1, -1, -1, -1] and copies.target.tolist() == [2, -1, -1, -1, -1]
    assert table.tolist() == [[4, 5, 6], [7, -1, 90], [4, 2, -1], [4, -1, -1], [7, -1, -1], [4, 5, 6]]
    assert shares.tolist() == [0] * 4 + [3, 1, 1, 1] + [0] * 4 and int(taken) == 3
    assert dec.status() == sar.TOPK_DEV_BLOCKS_EXHAUSTED | sar.TOPK_DEV_BAD_BLOCK


def test_free_limits(dec):
    table = ints([[3, -1, 50], [4, 5, 6], [7, 8, -1]])
    shares, free, taken = ints([0] * 10), ints([0, 1, 2, 9]), ints([3])
    dec.free_pages(ints([0, 7, -1, 1, 0]), table, shares, free, taken)
    # four pages come back where three were taken: the first is dropped; page 50 is none
    assert free.tolist() == [4, 5, 6, 9] and int(taken) == 0 and table.tolist() == [[-1] * 3, [-1] * 3, [7, 8, -1]]
    assert dec.status() == sar.TOPK_DEV_BLOCKS_EXHAUSTED | sar.TOPK_DEV_BAD_BLOCK


def test_compact_leaves_pages_of_others_and_takes_wrong_ones_off_the_list(dec):
    # 0 and 7 belong to someone else; 3 is free and named; 2 is listed twice; 70 is none
    table, shares, free, taken = ints([[9, 3, -1], [5, 9, -1]]), ints([0, 0, 0, 0, 0, 2, 0, 0, 0, 1]), ints([8, 4, 2, 1, 3, 2, 70]), ints([1])
    out = dec.compact_pages(table, shares, free, taken, 4)
    assert out.source.tolist() == [9, 5, -1, -1] and out.target.tolist() == [1, 2, -1, -1]
    assert table.tolist() == [[1, 3, -1], [2, 1, -1]] and shares.tolist() == [0, 1, 2, 0, 0, 0, 0, 0, 0, 0]
    assert int(taken) == 4 and free.tolist()[4:] == [4, 5, 9] and dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_nothing_to_do(dec):
    table, shares, free, taken = ints([[1, -1]]), ints([0] * 4), ints([0, 2, 3]), ints([0])
    dec.fork_pages(ints([]), ints([]), ints([]), table, shares, free, taken, 4)
    dec.free_pages(ints([]), table, shares, free, taken)
    assert dec.compact_pages(table[:0], shares[:0], free[:0], taken, 0).source.shape == (0,)
    dec.copy_pages([], sar.PageCopies(ints([0]), ints([1])))
    dec.copy_pages([torch.zeros(2, 3, device="cuda")], sar.PageCopies(ints([]), ints([])))
    assert table.tolist() == [[1, -1]] and int(taken) == 0
    ok(dec)


# ---- contents ----------------------------------------------------------------------------------------------------

def caches_of(pages):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return [r(pages, 16, 4, 128).bfloat16(),                     # pages in one piece
            r(pages, 4, 16, 64).half().transpose(1, 2),          # heads before tokens: in one piece as well
            r(pages, 16, 2, 3, 64).half()[:, :, :, 1],           # between other things
            r(pages, 16, 2, 72).half()[:, 3:14, 1, 4:],          # runs of 8 bytes' alignment
            r(pages, 33),                                        # scales, an odd number of bytes' pieces
            r(pages, 5, 7).to(torch.float8_e4m3fn),              # 35 bytes a page
            r(pages, 9, 6).half()[:, :, 1:4],                    # runs of 6 bytes
            r(pages, 4, 128).bfloat16(),
            (r(pages + 3, 700, 8) * 99).int()[3:],               # more than a chunk
            r(pages, 6, 6).half()[:, ::2, ::3],                  # no two elements side by side
            r(2 * pages, 8).half()[::2],
            r(pages, 16, 8).double().transpose(0, 1)[3]]


def test_copies_of_every_layout(dec):
    pages, rng = 60, random.Random(2)
    caches = caches_of(pages)
    backs = [c._base if c._base is not None else c for c in caches]
    order = rng.sample(range(pages), pages)
    source, target = [order[i % 20] for i in range(30)] + [-1, order[0]], order[25:55] + [order[59], -1]
    want = []
    for c in caches:
        base = c._base if c._base is not None else c
        copy = base.clone()
        view = copy.as_strided(c.shape, c.stride(), c.storage_offset())
        pairs = [(s, t) for s, t in zip(source, target) if s >= 0 and t >= 0]
        for s, t in pairs:
            view[t] = view[s].clone()
        want.append(copy)
    dec.copy_pages(caches, sar.PageCopies(ints(source), ints(target)))
    for i, (b, w) in enumerate(zip(backs, want)):
        assert torch.equal(b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b, w.view(torch.uint8) if w.dtype == torch.float8_e4m3fn else w), i
    ok(dec)


def test_copies_of_many_caches_kept_together(dec):
    caches = [torch.randn(30, 8 + i % 5, 16, device="cuda").half() for i in range(100)]
    want = [c.clone() for c in caches]
    kept = dec.page_caches(caches)
    for shift in range(3):
        source, target = [i for i in range(9)], [10 + shift * 5 + i for i in range(9)]
        dec.copy_pages(kept, sar.PageCopies(ints(source), ints(target)))
        for w in want:
            w[target] = w[source]
    assert all(torch.equal(a, b) for a, b in zip(caches, want))
    ok(dec)


def test_copies_outside_a_cache(dec):
    a, b = torch.arange(10.0, device="cuda")[:, None].repeat(1, 4), torch.arange(5.0, device="cuda")[:, None].repeat(1, 4)
    dec.copy_pages([a, b], sar.PageCopies(ints([7, 1, 1]), ints([2, 8, 99])))
    assert a[:, 0].tolist() == [0, 1, 7, 3, 4, 5, 6, 7, 1, 9] and b[:, 0].tolist() == [0, 1, 2, 3, 4]
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_copies_past_32_bits(dec):
    # elements of a cache whose offsets need more than 32 bits
    cache = torch.zeros(70, 1 << 26, dtype=torch.uint8, device="cuda")
    cache[3] = 7
    dec.copy_pages([cache], sar.PageCopies(ints([3]), ints([69])))
    assert int(cache[69].min()) == 7 and int(cache[:3].max()) == 0 and int(cache[68].max()) == 0
    ok(dec)


# ---- all of them together ------------------------------------------------------------------------------------------

def test_a_prompt_forked_decoded_freed_and_compacted(dec):
    """A prompt, eight samples of it, decode steps with attention that reads the prompt once, samples dropped and drawn anew,
    and the pool compacted: every step's attention is that of each request's own tokens, kept on the host."""
    g = torch.Generator().manual_seed(3)
    block, kv, heads, dk, rows, columns, pages = 16, 2, 8, 64, 10, 24, 200
    k = torch.full((pages, block, kv, dk), math.nan, device="cuda").half()
    v, means = k.clone(), torch.zeros(pages, kv, dk, device="cuda").half()
    table = torch.full((rows, columns), -1, dtype=torch.int32, device="cuda")
    shares, free, taken = ints([0] * pages), torch.randperm(pages, generator=g).int().cuda(), ints([0])
    told = [torch.zeros(0, 2, kv, dk).half() for _ in range(rows)]  # each request's keys and values
    kept = dec.page_caches([k, v, means])

    def grow(new):
        """Brings new[r] tokens to each request."""
        context = ints([len(t) for t in told])
        m = dec.kv_map(context, ints(new), table, free, taken, block, sum(new))
        fresh = torch.randn(sum(new), 2, kv, dk, generator=g).half()
        k.view(-1, kv, dk)[m.slots], v.view(-1, kv, dk)[m.slots] = fresh[:, 0].cuda(), fresh[:, 1].cuda()
        dec.block_means(k, table, context, ints(new), means)
        at = 0
        for r, n in enumerate(new):
            told[r] = torch.cat([told[r], fresh[at:at + n]])
            at += n

    def fork(parents, children, lens):
        copies = dec.fork_pages(ints(parents), ints(children), ints(lens), table, shares, free, taken, block)
        dec.copy_pages(kept, copies)
        for a, b, n in zip(parents, children, lens):
            told[b] = told[a][:n].clone()

    def release(requests):
        dec.free_pages(ints(requests), table, shares, free, taken)
        for r in requests:
            told[r] = told[r][:0]

    def check(prefix_of, prefix_lens, prefix_rows):
        lengths = [len(t) for t in told]
        q = torch.randn(rows, heads, dk, generator=g).half()
        out, lse = dec.shared_attention(q.cuda(), k, table, ints(lengths), ints(prefix_of), ints(prefix_lens), table[prefix_rows].contiguous(), v_cache=v, return_lse=True)
        width = max(lengths)
        own_k, own_v = torch.zeros(rows, width, kv, dk).half(), torch.zeros(rows, width, kv, dk).half()
        for r, t in enumerate(told):
            own_k[r, :len(t)], own_v[r, :len(t)] = t[:, 0], t[:, 1]
        want = pu.attention64(q, own_k, own_v, dk, torch.arange(rows, dtype=torch.int32)[:, None], lengths, list(range(rows)), width, dk ** -0.5)
        pu.check_attention(out, lse, (want[0], want[1], want[2] * 2.1, want[3] + 1e-5), torch.float16)
        # and attention over every block of the table, chosen by scores, is the same
        scores, lens = dec.block_scores(q.cuda(), means, table, ints(lengths), block)
        chosen = sar.Selector(0)(scores.flatten(0, 1), lens.flatten(), columns).view(rows, kv, columns)
        out, lse = dec.block_attention(q.cuda(), k, table, ints(lengths), chosen, v_cache=v, return_lse=True)
        pu.check_attention(out, lse, want, torch.float16)
        ok(dec)

    prompt = 101
    grow([prompt] + [0] * (rows - 1))
    fork([0] * 8, list(range(1, 9)), [prompt] * 8)
    for _ in range(3):
        grow([0] + [1 + r % 3 for r in range(8)] + [0])
        check([0] * 9 + [-1], [prompt], [0])
    release([2, 5, 9, 7])
    fork([3, 3, 1], [2, 5, 9], [len(told[3]), len(told[3]), 110 if len(told[1]) >= 110 else len(told[1])])
    grow([0, 2, 30, 1, 40, 3, 1, 0, 20, 9])
    check([0, 0, 0, 0, 0, 0, 0, -1, 0, 0], [prompt], [0])
    release([0, 4])
    moves = dec.compact_pages(table, shares, free, taken, 50)
    dec.copy_pages(kept, moves)
    live = sorted({p for row in table.tolist() for p in row if p >= 0})
    assert live == list(range(len(live))) and int((moves.source >= 0).sum()) > 0
    check([-1, 0, 0, 0, -1, 0, 0, -1, 0, 0], [prompt], [1])
    grow([50, 1, 1, 1, 0, 1, 1, 7, 1, 1])
    check([-1, 0, 0, 0, -1, 0, 0, -1, 0, 0], [96], [1])
    release(list(range(rows)))
    assert int(taken) == 0 and sorted(free.tolist()) == list(range(pages)) and not shares.any() and (table == -1).all()
    ok(dec)


@pytest.mark.parametrize("kw", [dict(), dict(prompts=3, samples=9, tokens=700, heads=32, kv_heads=8, dim=128, block=64, topk=4), dict(prompts=1, samples=1, tokens=40, steps=1, heads=1, kv_heads=1, block=33),
                                dict(prompts=4, samples=2, tokens=129, block=1, heads=6, kv_heads=3, topk=40)])
def test_example_of_shared_prompts(dec, kw):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompts.py")
    spec = importlib.util.spec_from_file_location("shared_prompts", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # half steps of bf16 for the probabilities, the part behind the prefix and the result, of values below 5
    assert example.run(**kw) < 3 * 2.0 ** -8 * 5
