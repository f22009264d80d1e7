"""Blocks, shared prefixes and pages where they went wrong once."""
import random

import pytest
import torch

import sparse_attention_row_gb300 as sar
from tests import test_blocks_gpu as blocks
from tests import test_pages_gpu as pages
from tests import test_shared_gpu as shared
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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("next_n", [3, 4, 5])
@pytest.mark.parametrize("heads, kv, dk", [(8, 8, 376), (8, 8, 384), (14, 7, 432), (6, 6, 504), (12, 6, 512), (24, 12, 512), (9, 9, 400), (5, 5, 576)])
def test_scores_of_few_rows_whose_queries_fill_a_ctas_shared_memory(dec, next_n, heads, kv, dk):
    lengths = [max(0, b + j) for b in (70, 0, 300) for j in range(next_n)]
    requests = [r // next_n for r in range(len(lengths))]
    case = blocks.scores_case(20, lengths, requests, heads, kv, dk, torch.bfloat16, 4)
    blocks.check_scores(dec, case, lengths, requests, 4, sinks=1, recent=1, next_n=next_n)
    blocks.check_scores(dec, case, lengths, requests, 4, row_request=True)
    assert dec.status() == 0


def test_fork_enters_no_free_page_that_is_none(dec):
    # 12 and -4 are no pages of the pool; they are taken off the list all the same
    table = ints([[4, 5], [-1, -1], [-1, -1], [-1, -1], [-1, -1]])
    shares, free, taken = ints([0] * 12), ints([12, 3, -4]), ints([0])
    copies = dec.fork_pages(ints([0, 0, 0, 0]), ints([1, 2, 3, 4]), ints([5, 6, 7, 4]), table, shares, free, taken, 4)
    assert copies.source.tolist() == [-1, 5, -1, -1] and copies.target.tolist() == [-1, 3, -1, -1]
    assert table.tolist() == [[4, 5], [4, -1], [4, 3], [4, -1], [4, -1]] and int(taken) == 3
    assert shares.tolist() == [0] * 4 + [4] + [0] * 7 and dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_prefixes_that_are_none_are_reported_whichever_way_a_call_takes(dec):
    # the third request names a prefix that there is none of, and has no rows
    lengths, requests = [40, 50, 33], [0, 1, 3]
    case = shared.make(30, [32], [0, 0, -1, 0], lengths, requests, 4, 1, 64, 64, False, torch.float16, 16)
    shared.check(dec, case, [32], [0, 0, 1, 0], lengths, requests, 64, 16, allowed=sar.TOPK_DEV_BAD_BLOCK, row_request=ints(requests))
    q, k, v, hidden, whole, prefix_table = case
    for table in shared.tables(q, k, v, 64, prefix_table, 16):
        for third, bits in ((1, sar.TOPK_DEV_BAD_BLOCK), (0, 0), (-2 ** 31, 0), (2 ** 31 - 1, sar.TOPK_DEV_BAD_BLOCK)):
            dec.reset()
            dec.shared_attention(q.cuda(), k.cuda(), hidden.cuda(), ints(lengths), ints([0, 0, third, 0]), ints([32]), table.cuda(), v_cache=v.cuda(), row_request=ints(requests))
            assert dec.status() == bits


@pytest.mark.parametrize("by_row", [False, True])
def test_who_reads_the_prefix_of_a_request_with_a_row_that_sees_less(dec, by_row):
    # the request's own row of the table names other pages than its prefix, and its second row sees less than that holds
    g = torch.Generator().manual_seed(31)
    q, k, v = (torch.randn(s, generator=g).half() for s in ((2, 4, 64), (8, 16, 2, 64), (8, 16, 2, 64)))
    own, prefix = torch.tensor([[1, 2, 3]], dtype=torch.int32), torch.tensor([[6, 5]], dtype=torch.int32)
    lengths, mixed = [40, 20], torch.tensor([[6, 5, 3], [1, 2, 3]], dtype=torch.int32)
    want = blocks.pu.attention64(q, k, v, 64, mixed if by_row else own.expand(2, -1), lengths, [0, 1], 16, 64 ** -0.5)
    room = want[0], want[1], want[2] * 2.1, want[3] + 1e-5  # the part behind the prefix is rounded once more
    for table in shared.tables(q, k, v, 64, prefix, 16):
        out, lse = dec.shared_attention(q.cuda(), k.cuda(), own.cuda(), ints(lengths), ints([0]), ints([32]), table.cuda(), v_cache=v.cuda(), return_lse=True,
                                        **(dict(row_request=ints([0, 0])) if by_row else dict(next_n=2)))
        blocks.pu.check_attention(out, lse, room, torch.float16)
    assert dec.status() == 0


@pytest.mark.parametrize("rows, listed", [(3000, 1024), (3000, 1025), (900, 5000), (30000, 40000), (500000, 60000), (500000, 45), (250000, 16 * 1024 + 1)])
def test_requests_that_are_listed_twice_among_many(dec, rows, listed):
    # anywhere in the list, some next to each other, some that are none; pages that several rows hold
    rng = random.Random(listed)
    pool = pages.Pool(rows, 1, rows, 4, rng)
    owners = rows - rows // 3
    pool.table, pool.taken = [[p] for p in pool.free[:owners]], owners
    for r in range(owners, rows):
        pool.table.append(list(rng.choice(pool.table[:200])))
        pool.shares[pool.table[r][0]] += 1
    gone = rng.choices(range(rows), k=listed - 4)
    for at in (0, 7, len(gone) // 2, len(gone)):
        gone.insert(at, gone[max(at - 1, 0)])
    state = pool.device()
    bad = list(gone)
    bad[3:3] = [-1, rows, -2 ** 31, 2 ** 31 - 1, rows, -1]
    dec.free_pages(ints(bad), *state)
    pool.release(gone)
    pool.same(state)
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_time_to_free_grows_with_the_number_of_requests(dec):
    # a quarter of the most that a call takes: compared one with another they would take some hundred milliseconds
    n = 1 << 18
    rows = torch.randperm(n, device="cuda", dtype=torch.int32)
    held = rows.tolist()  # the table is these numbers' memory
    table, shares, free, taken = rows[:, None], torch.zeros_like(rows), torch.zeros_like(rows), ints([n])
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    listed = torch.randint(0, n, (n,), device="cuda", dtype=torch.int32)
    dec.free_pages(ints([0]), ints([[-1]]), ints([0]), ints([0]), ints([1]))  # the kernel is loaded with its first launch
    torch.cuda.synchronize()
    start.record()
    dec.free_pages(listed, table, shares, free, taken)
    end.record()
    end.synchronize()
    assert start.elapsed_time(end) < 20
    first = list(dict.fromkeys(listed.tolist()))
    assert int(taken) == n - len(first) and free[n - len(first):].tolist() == [held[r] for r in first]
    assert not shares.any() and int((table < 0).sum()) == len(first) and dec.status() == 0


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_recent_blocks_keep_what_follows_a_row_out_of_its_scores(dec, rows):
    # a piece's rows, whose requests' last pages hold one to some tokens more than they see
    block, lengths = 8, [31 + r for r in range(rows)]
    q, more = torch.randn(rows, 4, 64).half(), lengths[-1] + 5
    k = torch.randn(16, block, 2, 64).half().cuda()
    table = torch.randperm(16)[None].int().cuda()
    scores = []
    for follows in (0.0, 100.0):  # the tokens behind each row, of its own last block
        for r in range(rows):
            cache = k.clone()
            t = torch.arange(lengths[r], more)
            cache[table[0, t // block].long(), t % block] = follows
            means = dec.block_means(cache, table, ints([0]), ints([more]), torch.zeros(16, 2, 64).half().cuda())
            out = torch.zeros(rows, 2, 16, device="cuda")
            dec.block_scores(q.cuda(), means, table, ints(lengths), block, recent_blocks=1, next_n=rows, out=out)
            scores.append(out[r])
    assert torch.equal(torch.stack(scores[:rows]), torch.stack(scores[rows:])) and dec.status() == 0
