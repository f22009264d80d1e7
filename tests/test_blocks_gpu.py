"""Blocks chosen by a cheap score: means, scores and attention against their definitions in 64 bits."""
import math

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


# ---- means -----------------------------------------------------------------------------------------------------

def means64(k, table, context, new, block, means):
    """(means, bound of their error before the last rounding); pages that got no token keep what they had."""
    want, room = means.double(), torch.zeros(means.shape, dtype=torch.float64)
    for r, (c, n) in enumerate(zip(context, new)):
        c, n = max(c, 0), max(n, 0)
        for col in range(c // block, (c + n - 1) // block + 1) if n else []:
            page, held = int(table[r, col]), min(block, c + n - col * block)
            x = k[page, :held].double()
            want[page], room[page] = x.mean(0), x.abs().mean(0) * (held + 2) * pu.ACC
    return want, room


def check_means(got, want, room, dtype):
    got = got.cpu().double()
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-38  # half a step of the smallest numbers
    far, most = (got - want).abs(), room + want.abs() * pu.U[dtype] * (1 + 2.0 ** -6) + tiny
    assert torch.isfinite(got).all() and (far <= most).all(), f"{float((far / most).max()):.2f} of the bound off"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("block, kv, dk", [(64, 8, 128), (16, 1, 64), (1, 2, 8), (33, 3, 72), (128, 1, 576), (7, 5, 576), (256, 40, 128)])
def test_means(dec, dtype, block, kv, dk):
    g = torch.Generator().manual_seed(block + dk)
    context, new = [0, 5, 64, 100, 0, 200, 63, 1, 128], [1, 3, 1, 0, 300, 130, 2, 64, 0]
    total = [c + n for c, n in zip(context, new)]
    table, blocks = pu.block_table(g, total, block)
    k = pu.poisoned(torch.randn(blocks, block, kv, dk, generator=g).to(dtype), table, total, block)
    means = torch.randn(blocks, kv, dk, generator=g).to(dtype)
    want, room = means64(k, table, context, new, block, means)
    got = dec.block_means(k.cuda(), table.cuda(), ints(context), ints(new), means.cuda())
    check_means(got, want, room, dtype)
    untouched = room.flatten(1).amax(1) == 0
    assert torch.equal(got.cpu()[untouched], means[untouched])
    ok(dec)


def test_means_of_many_requests_and_strided_views(dec):
    # more requests than are summed up at a time; keys and means between other things
    g = torch.Generator().manual_seed(4)
    n, block = 2500, 8
    context = torch.randint(0, 20, (n,), generator=g).tolist()
    new = torch.randint(0, 4, (n,), generator=g).tolist()
    total = [c + m for c, m in zip(context, new)]
    table, blocks = pu.block_table(g, total, block, columns=6)
    big = torch.randn(blocks, 2, block, 5, 32, generator=g).half()
    k = big[:, 1, :, 1:3, 16:]
    wide = torch.randn(blocks, 3, 40, generator=g).half()
    want, room = means64(k, table, context, new, block, wide[:, ::2, 8:24])
    dev = wide.cuda()
    dec.block_means(big.cuda()[:, 1, :, 1:3, 16:], table.cuda(), ints(context), ints(new), dev[:, ::2, 8:24])
    check_means(dev[:, ::2, 8:24], want, room, torch.float16)
    assert torch.equal(dev[:, 1].cpu(), wide[:, 1]) and torch.equal(dev[:, :, :8].cpu(), wide[:, :, :8]) and torch.equal(dev[:, :, 24:].cpu(), wide[:, :, 24:])
    ok(dec)


def test_means_of_lengths_and_pages_that_are_none(dec):
    k = torch.ones(4, 4, 1, 8, device="cuda").half()
    means = torch.zeros(4, 1, 8, device="cuda").half()
    table = ints([[0, 1], [-1, 9], [2, 3]])
    dec.block_means(k, table, ints([-7, 0, 5]), ints([3, 8, -2]), means)  # a negative length reads as 0
    assert means[:, 0, 0].tolist() == [1, 0, 0, 0] and dec.status() == sar.TOPK_DEV_BAD_BLOCK
    dec.reset()
    dec.block_means(k, table, ints([0, 0, 6]), ints([0, 0, 2 ** 31 - 1]), means)  # the table ends
    assert means[:, 0, 0].tolist() == [1, 0, 0, 1] and dec.status() == sar.TOPK_DEV_TABLE_FULL
    dec.block_means(k, table[:0], ints([]), ints([]), means)


def test_means_propagate_infinities_and_nan(dec):
    k = torch.zeros(1, 8, 1, 8).half()
    k[0, 2, 0, 0], k[0, 3, 0, 1], k[0, 1, 0, 2], k[0, 4, 0, 2], k[0, 7, 0, 3] = math.inf, math.nan, math.inf, -math.inf, math.nan
    got = dec.block_means(k.cuda(), ints([[0]]), ints([0]), ints([7]), torch.zeros(1, 1, 8, device="cuda").half()).cpu()[0, 0]
    assert got[0] == math.inf and got[1].isnan() and got[2].isnan() and (got[3:] == 0).all()


# ---- scores ----------------------------------------------------------------------------------------------------

def scores64(q, means, table, lengths, requests, block, sinks, recent, columns):
    """(scores with nan past each row's blocks, bound of their error, blocks of each row)."""
    rows, heads, dk = q.shape
    kv = means.shape[1]
    out = torch.full((rows, kv, columns), math.nan, dtype=torch.float64)
    tol, lens = out.clone(), []
    for r in range(rows):
        n = min(-(-int(lengths[r]) // block), columns)
        lens.append(n)
        m = means[table[requests[r], :n].long()].double()
        qq = q[r].double().view(kv, heads // kv, dk)
        out[r, :, :n] = torch.einsum("gd,jgd->gj", qq.sum(1), m)
        tol[r, :, :n] = torch.einsum("gd,jgd->gj", qq.abs().sum(1), m.abs()) * (heads // kv + dk + 4) * pu.ACC + 1e-30
        out[r, :, :min(sinks, n)] = math.inf
        out[r, :, max(0, n - recent):n] = math.inf
    return out, tol, lens


def scores_case(seed, lengths, requests, heads, kv, dk, dtype, block):
    g = torch.Generator().manual_seed(seed)
    longest = [max([n for n, b in zip(lengths, requests) if b == i] + [0]) for i in range(max(requests) + 1)]
    table, blocks = pu.block_table(g, longest, block)
    means = torch.full((blocks, kv, dk), math.nan).to(dtype)
    used = table[table >= 0].long()
    means[used] = torch.randn(len(used), kv, dk, generator=g).to(dtype)
    return torch.randn(len(lengths), heads, dk, generator=g).to(dtype), means, table


def check_scores(dec, case, lengths, requests, block, sinks=0, recent=0, next_n=None, row_request=False, columns=None):
    q, means, table = case
    columns = columns or table.shape[1]
    want, tol, lens = scores64(q, means, table, lengths, requests, block, sinks, recent, columns)
    out = torch.full(want.shape, 7.25, device="cuda")
    got, got_lens = dec.block_scores(q.cuda(), means.cuda(), table.cuda(), ints(lengths), block, sink_blocks=sinks, recent_blocks=recent, next_n=next_n,
                                     row_request=ints(requests) if row_request else None, out=out)
    assert got.data_ptr() == out.data_ptr() and got_lens.tolist() == [[n] * means.shape[1] for n in lens]
    got = got.cpu().double()
    past = want.isnan()
    assert (got[past] == 7.25).all(), "written past a row's blocks"
    top = want == math.inf
    assert (got[top] == math.inf).all()
    rest = ~past & ~top
    far = (got - want).abs()[rest]
    assert (far <= tol[rest]).all(), f"{float((far / tol[rest]).max()):.2f} of the bound off"


LENGTHS = [0, 1, 64, 65, 1000, 0, 4000, 17, 8200]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads, kv, dk, block", [(64, 8, 128, 64), (8, 8, 64, 16), (5, 1, 8, 33), (24, 3, 72, 7), (128, 1, 576, 16), (32, 4, 128, 1)])
def test_scores(dec, dtype, heads, kv, dk, block):
    requests = list(range(len(LENGTHS)))
    check_scores(dec, scores_case(1, LENGTHS, requests, heads, kv, dk, dtype, block), LENGTHS, requests, block, sinks=1, recent=2)
    check_scores(dec, scores_case(2, LENGTHS, requests, heads, kv, dk, dtype, block), LENGTHS, requests, block)
    ok(dec)


@pytest.mark.parametrize("next_n", [2, 3, 5, 9, 16, 17, 40])
def test_scores_of_rows_of_a_request(dec, next_n):
    lengths = [max(0, b + j) for b in (300, 0, 2500) for j in range(next_n)]
    lengths[next_n + 1] = 0
    requests = [r // next_n for r in range(len(lengths))]
    case = scores_case(3, lengths, requests, 16, 2, 128, torch.bfloat16, 16)
    check_scores(dec, case, lengths, requests, 16, sinks=2, recent=1, next_n=next_n)
    check_scores(dec, case, lengths, requests, 16, recent=500, row_request=True)
    check_scores(dec, case, lengths, requests, 16, sinks=3, row_request=True, columns=None)
    ok(dec)


@pytest.mark.parametrize("heads, kv, dk", [(6, 2, 128), (24, 1, 64), (25, 1, 256), (75, 3, 40), (64, 4, 128), (4, 4, 8), (2, 1, 248), (26, 1, 64), (16, 2, 264)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_scores_of_many_rows_of_a_request(dec, heads, kv, dk, dtype):
    # groups that fill the columns and that do not, pages that there are none of, rows that see nothing among others
    rows = 150
    lengths = [0 if r % 11 == 5 else 300 + 7 * r for r in range(rows)]
    case = scores_case(8, lengths, [0] * rows, heads, kv, dk, dtype, 2)
    check_scores(dec, case, lengths, [0] * rows, 2, sinks=2, recent=3, next_n=rows)
    requests = [0] * 70 + [1] * 3 + [2] * 77
    case = scores_case(9, lengths, requests, heads, kv, dk, dtype, 4)
    check_scores(dec, case, lengths, requests, 4, recent=1, row_request=True)
    ok(dec)
    q, means, table = case
    table = table.clone()
    bad = [3, 7, 130]
    table[0, 3], table[0, 7], table[2, 130] = -5, means.shape[0], 2 ** 31 - 1
    good = table.clamp(0, means.shape[0] - 1)
    want, tol, _ = scores64(q, torch.nan_to_num(means.float()).to(dtype), good, lengths, requests, 4, 0, 0, table.shape[1])
    got, _ = dec.block_scores(q.cuda(), means.cuda(), table.cuda(), ints(lengths), 4, row_request=ints(requests))
    got = got.cpu().double()
    for r, b in enumerate(requests):
        n = -(-lengths[r] // 4)
        off = torch.tensor([bool((table[b, j] < 0) | (table[b, j] >= means.shape[0])) for j in range(n)], dtype=torch.bool)
        assert (got[r, :, :n][:, off] == -math.inf).all()
        assert ((got[r, :, :n] - want[r, :, :n]).abs() <= tol[r, :, :n])[:, ~off].all()
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


@pytest.mark.parametrize("next_n", [2, 3, 4, 6])
@pytest.mark.parametrize("heads, kv", [(32, 1), (64, 2), (33, 1), (66, 2), (6, 2), (28, 4), (4, 2), (2, 2)])
def test_scores_of_a_few_rows_of_a_request(dec, next_n, heads, kv):
    # about the smallest tiles that the tensor cores take, of groups with and without a kernel of their own, and too large ones
    lengths = [max(0, b + j) for b in (4100, 0, 1, 900) for j in range(next_n)]
    lengths[0] = 17
    requests = [r // next_n for r in range(len(lengths))]
    case = scores_case(14, lengths, requests, heads, kv, 128, torch.float16, 8)
    check_scores(dec, case, lengths, requests, 8, sinks=1, recent=2, next_n=next_n)
    check_scores(dec, case, lengths, requests, 8, sinks=1, row_request=True)
    ok(dec)


def test_scores_that_are_no_numbers_stay_in_their_blocks(dec):
    for rows in (1, 9):
        means = torch.zeros(300, 1, 64).half()
        means[5, 0, 0], means[130, 0, 1], means[131, 0, 2] = math.inf, math.nan, -math.inf
        got, _ = dec.block_scores(torch.ones(rows, 4, 64).half().cuda(), means.cuda(), torch.arange(300, dtype=torch.int32, device="cuda")[None], ints([300] * rows), 1, next_n=rows)
        got = got.cpu()[:, 0]
        assert (got[:, 5] == math.inf).all() and got[:, 130].isnan().all() and (got[:, 131] == -math.inf).all()
        assert (got[:, [i for i in range(300) if i not in (5, 130, 131)]] == 0).all()


def test_scores_with_a_request_for_each_row(dec):
    requests = [0] * 9 + [2] * 3 + [1] + [2] * 2 + [3, 0, 3]
    lengths = [200 + i for i in range(9)] + [0, 130, 600, 1, 128, 129, 77, 900, 2]
    check_scores(dec, scores_case(5, lengths, requests, 6, 2, 64, torch.float16, 4), lengths, requests, 4, recent=1, row_request=True)


def test_scores_of_padding_rows_bad_lengths_and_pages(dec):
    q, means, table = scores_case(6, [100, 64], [0, 1], 4, 1, 64, torch.float16, 16)
    q = q.repeat(2, 1, 1)
    out = torch.full((4, 1, 3), 7.25, device="cuda")
    got, lens = dec.block_scores(q.cuda(), means.cuda(), table.cuda(), ints([100, 50, -3, 2 ** 31 - 1]), 16, row_request=ints([0, -1, 1, -1]), out=out)
    # columns past the output's are neither scored nor counted; a negative request sees nothing
    assert lens.flatten().tolist() == [3, 0, 0, 0] and (got[1:] == 7.25).all() and (got[0] != 7.25).all()
    assert dec.status() == sar.TOPK_DEV_LENGTH_CLAMPED
    dec.reset()
    table[0, 1], table[0, 2] = -1, means.shape[0]
    got, lens = dec.block_scores(q.cuda(), means.cuda(), table.cuda(), ints([100, 50, 100, 0]), 16, sink_blocks=2, row_request=ints([0, -1, 0, 1]))
    assert lens.flatten().tolist() == [7, 0, 7, 0] and got[0, 0, 0] == math.inf and (got[0, 0, 1:3] == -math.inf).all() and got[0, 0, 3:].isfinite().all()
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_scores_strided_views(dec):
    lengths, requests = [70, 200, 15], [0, 1, 2]
    q, means, table = scores_case(7, lengths, requests, 6, 2, 64, torch.bfloat16, 16)
    big_q, big_m = torch.randn(3, 12, 96).bfloat16(), torch.randn(means.shape[0], 4, 96).bfloat16()
    big_q[:, ::2, 32:], big_m[:, 1::2, :64] = q, means
    out = torch.full((3, 5, 40), 7.25, device="cuda")
    got, _ = dec.block_scores(big_q.cuda()[:, ::2, 32:], big_m.cuda()[:, 1::2, :64], table.cuda(), ints(lengths), 16, out=out[:, 1:4:2, 3:20])
    want, tol, _ = scores64(q, means, table, lengths, requests, 16, 0, 0, 17)
    past = want.isnan()
    got = got.cpu().double()
    assert (got[past] == 7.25).all() and ((got - want).abs()[~past] <= tol[~past]).all()
    assert (out[:, ::2] == 7.25).all() and (out[:, :, :3] == 7.25).all() and (out[:, :, 20:] == 7.25).all()


# ---- attention over chosen blocks --------------------------------------------------------------------------------

def blocks64(q, k, v, dv, table, lengths, requests, block, scale, chosen):
    """As attention64, with a list of blocks for each row and key-value head."""
    kv = k.shape[2]
    group = q.shape[1] // kv
    parts = []
    for h in range(kv):
        index = torch.where(chosen[:, h, :, None] >= 0, chosen[:, h, :, None].long() * block + torch.arange(block), -1).flatten(1)
        parts.append(pu.attention64(q[:, h * group:(h + 1) * group], k[:, :, h:h + 1], None if v is None else v[:, :, h:h + 1], dv, table, lengths, requests, block, scale, indices=index))
    return tuple(torch.cat(x, 1) for x in zip(*parts))


def blocks_case(seed, lengths, requests, heads, kv, dk, dv, latent, dtype, block, chosen):
    g = torch.Generator().manual_seed(seed)
    longest = [max([n for n, b in zip(lengths, requests) if b == i] + [0]) for i in range(max(requests) + 1)]
    table, blocks = pu.block_table(g, longest, block)
    k = pu.poisoned(torch.randn(blocks, block, kv, dk, generator=g).to(dtype), table, longest, block)
    v = None if latent else pu.poisoned(torch.randn(blocks, block, kv, dv, generator=g).to(dtype), table, longest, block)
    lists = torch.full((len(lengths), kv, chosen), -1, dtype=torch.int32)
    for r, n in enumerate(lengths):
        used = -(-n // block)
        for h in range(kv):
            pick = torch.randperm(used, generator=g)[:chosen]
            lists[r, h, torch.randperm(chosen, generator=g)[:len(pick)]] = pick.int()  # -1 anywhere
    return torch.randn(len(lengths), heads, dk, generator=g).to(dtype), k, v, table, lists


def run_blocks(dec, case, lengths, lists=None, **kw):
    q, k, v, table, chosen = case
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    return dec.block_attention(q.cuda(), k.cuda(), table.cuda(), ints(lengths), c(chosen) if lists is None else lists, v_cache=c(v), return_lse=True, **kw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads, kv, dk, dv, latent, block, chosen", [
    (64, 8, 128, 128, False, 64, 4), (4, 4, 64, 64, False, 16, 9), (12, 1, 128, 64, False, 32, 1), (6, 2, 72, 40, False, 33, 5), (16, 1, 576, 512, True, 64, 3),
    (128, 1, 576, 512, True, 16, 10), (3, 3, 8, 8, False, 1, 200), (8, 2, 256, 256, False, 200, 2), (8, 2, 64, 128, False, 7, 31)])
def test_block_attention(dec, dtype, heads, kv, dk, dv, latent, block, chosen):
    lengths = [0, 1, 64, 129, 700, 0, 333, 1500]
    requests = list(range(len(lengths)))
    case = blocks_case(block, lengths, requests, heads, kv, dk, dv, latent, dtype, block, chosen)
    out, lse = run_blocks(dec, case, lengths, v_dim=dv)
    q, k, v, table, lists = case
    pu.check_attention(out, lse, blocks64(q, k, v, dv, table, lengths, requests, block, dk ** -0.5, lists), dtype)
    ok(dec)


@pytest.mark.parametrize("next_n", [2, 5])
def test_block_attention_of_rows_of_a_request(dec, next_n):
    lengths = [b + j for b in (200, 0, 63, 900) for j in range(next_n)]
    requests = [r // next_n for r in range(len(lengths))]
    case = blocks_case(9, lengths, requests, 8, 2, 128, 128, False, torch.bfloat16, 32, 6)
    q, k, v, table, lists = case
    want = blocks64(q, k, v, 128, table, lengths, requests, 32, 128 ** -0.5, lists)
    pu.check_attention(*run_blocks(dec, case, lengths, next_n=next_n), want, torch.bfloat16)
    pu.check_attention(*run_blocks(dec, case, lengths, row_request=ints(requests)), want, torch.bfloat16)
    ok(dec)


def test_block_attention_many_rows(dec):
    # more units than CTAs: runs of whole units, and splits where few are long
    lengths = [1 + (37 * i) % 600 for i in range(400)]
    requests = [i % 7 for i in range(400)]
    case = blocks_case(10, lengths, requests, 8, 2, 64, 64, False, torch.float16, 16, 12)
    q, k, v, table, lists = case
    want = blocks64(q, k, v, 64, table, lengths, requests, 16, 64 ** -0.5, lists)
    pu.check_attention(*run_blocks(dec, case, lengths, row_request=ints(requests)), want, torch.float16)
    ok(dec)


def test_block_attention_few_long_lists(dec):
    lengths = [20000, 15001]
    case = blocks_case(11, lengths, [0, 1], 4, 1, 128, 128, False, torch.bfloat16, 64, 250)
    q, k, v, table, lists = case
    want = blocks64(q, k, v, 128, table, lengths, [0, 1], 64, 128 ** -0.5, lists)
    pu.check_attention(*run_blocks(dec, case, lengths), want, torch.bfloat16)


def test_block_attention_lists_of_all_heads_and_strange_entries(dec):
    # one list for all heads of a row; blocks past the row's, out of all range, and one named twice, which counts twice
    lengths = [100, 300]
    case = blocks_case(12, lengths, [0, 1], 4, 2, 64, 64, False, torch.float16, 16, 6)
    q, k, v, table, _ = case
    lists = torch.tensor([[3, 900, 0, -5, 6, 2 ** 31 - 1], [18, 1, 1, 40, -1, 17]], dtype=torch.int32)
    both = lists[:, None].expand(2, 2, 6)
    inside = torch.where((both >= 0) & (both < 19), both, -1)
    want = blocks64(q, k, v, 64, table, lengths, [0, 1], 16, 0.3, inside)
    pu.check_attention(*run_blocks(dec, case, lengths, lists=lists.cuda(), scale=0.3), want, torch.float16)
    wide = torch.full((2, 3, 4, 8), 5, dtype=torch.int32, device="cuda")
    wide[:, 1, ::2, 1:7] = both.cuda()
    pu.check_attention(*run_blocks(dec, case, lengths, lists=wide[:, 1, ::2, 1:7], scale=0.3), want, torch.float16)
    ok(dec)


def test_block_attention_pages_outside_the_cache(dec):
    lengths = [160]
    case = blocks_case(13, lengths, [0], 2, 1, 64, 64, False, torch.float16, 16, 10)
    q, k, v, table, lists = case
    bad = table.clone()
    bad[0, 4], bad[0, 5] = -1, k.shape[0]
    out, lse = run_blocks(dec, (q, k, v, bad, lists), lengths)
    seen = torch.where((lists == 4) | (lists == 5), -1, lists)
    pu.check_attention(out, lse, blocks64(q, k, v, 64, table, lengths, [0], 16, 64 ** -0.5, seen), torch.float16)
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_block_attention_scores_that_are_no_numbers(dec):
    # a block of minus infinities is as if it were not there; a row with nothing else gets zeros
    lengths = [32, 16]
    q = torch.ones(2, 2, 64).bfloat16()
    k = torch.zeros(3, 16, 1, 64).bfloat16()
    k[0, :, 0, 0] = -math.inf
    v = torch.arange(3 * 16 * 64, dtype=torch.float32).view(3, 16, 1, 64).remainder(7).bfloat16()
    table, lists = torch.tensor([[0, 1], [0, -1]], dtype=torch.int32), torch.tensor([[[0, 1]], [[0, -1]]], dtype=torch.int32)
    out, lse = run_blocks(dec, (q, k, v, table, lists), lengths)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    want = v[1].double().mean(0)
    assert ((out[0].cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-6).all() and (lse[0] - math.log(16)).abs().max() < 1e-5


# ---- a step of all three with the selection ----------------------------------------------------------------------

def test_a_step_of_all(dec):
    g = torch.Generator().manual_seed(21)
    block, kv, heads, dk, topk = 16, 2, 8, 64, 5
    context, new = [0, 200, 77, 511, 16], [40, 1, 3, 2, 0]
    total = [c + n for c, n in zip(context, new)]
    table, blocks = pu.block_table(g, total, block)
    k = torch.randn(blocks, block, kv, dk, generator=g).half()
    v = torch.randn(blocks, block, kv, dk, generator=g).half()
    q = torch.randn(5, heads, dk, generator=g).half()
    sel = sar.Selector(0)
    c = lambda x: x.cuda()  # noqa: E731
    means = torch.zeros(blocks, kv, dk).half().cuda()
    dec.block_means(c(k), c(table), ints([0] * 5), ints(context), means)
    dec.block_means(c(k), c(table), ints(context), ints(new), means)
    scores, lens = dec.block_scores(c(q), means, c(table), ints(total), block, sink_blocks=1, recent_blocks=1)
    chosen = sel(scores.flatten(0, 1), lens.flatten(), topk).view(5, kv, topk)
    out, lse = dec.block_attention(c(q), c(k), c(table), ints(total), chosen, v_cache=c(v), return_lse=True)
    for r, n in enumerate(total):
        used = -(-n // block)
        for h in range(kv):
            got = sorted(x for x in chosen[r, h].tolist() if x >= 0)
            s = scores[r, h, :used]
            assert got == sorted(torch.sort(s, descending=True, stable=True).indices[:topk].tolist())
            assert len(got) == min(topk, used) and (used == 0 or (0 in got and used - 1 in got))
    pu.check_attention(out, lse, blocks64(q, k, v, dk, table, total, list(range(5)), block, dk ** -0.5, chosen.cpu()), torch.float16)
    ok(dec)
