"""Blocks, shared prefixes and pages where they went wrong once."""
import pytest
import torch

import sparse_attention_row_gb300 as sar
from tests import test_blocks_gpu as blocks
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
