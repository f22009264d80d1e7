"""Attention of requests that begin with the same pages, against the definition in 64 bits over each request's own tokens."""
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


def make(seed, prefixes, prefix_of, lengths, requests, heads, kv, dk, dv, latent, dtype, block):
    """prefixes: tokens of each; prefix_of: of each request; lengths, requests: of each row. The requests' table without the
    pages that they share (the call must not look at those), and the one with them."""
    g = torch.Generator().manual_seed(seed)
    longest = [max([n for n, b in zip(lengths, requests) if b == i] + [0]) for i in range(len(prefix_of))]
    full = [n // block for n in prefixes]
    shares = [0 <= p < len(prefixes) and all(n >= full[p] * block for n, b in zip(lengths, requests) if b == i) for i, p in enumerate(prefix_of)]
    own = [n - full[p] * block if s else n for n, p, s in zip(longest, prefix_of, shares)]
    used = [-(-max(n, 0) // block) for n in prefixes + own]
    order = torch.randperm(sum(used) + 2, generator=g).int().tolist()
    pages, at = [], 0
    for u in used:
        pages.append(order[at:at + u])
        at += u
    columns = max([-(-n // block) for n in longest] + [1])
    hidden, whole = torch.full((len(prefix_of), columns), -7, dtype=torch.int32), torch.full((len(prefix_of), columns), -1, dtype=torch.int32)
    for i, (p, s) in enumerate(zip(prefix_of, shares)):
        mine = pages[len(prefixes) + i]
        n = full[p] if s else 0
        hidden[i, n:n + len(mine)] = whole[i, n:n + len(mine)] = torch.tensor(mine, dtype=torch.int32)
        if n:
            whole[i, :n] = torch.tensor(pages[p][:n], dtype=torch.int32)
    prefix_table = torch.full((max(len(prefixes), 1), max(used[:len(prefixes)] + [1])), -1, dtype=torch.int32)
    for i, u in enumerate(pages[:len(prefixes)]):
        prefix_table[i, :len(u)] = torch.tensor(u, dtype=torch.int32)
    total = sum(used) + 2
    k = torch.randn(total, block, kv, dk, generator=g).to(dtype)
    v = None if latent else torch.randn(total, block, kv, dv, generator=g).to(dtype)
    # what no one sees is NaN: pages of no one, and behind each request's last token
    keep = torch.zeros(total, block, dtype=torch.bool)
    for i, n in enumerate(longest):
        t = torch.arange(n)
        keep[whole[i, t // block].long(), t % block] = True
    k = torch.where(keep[..., None, None], k, math.nan)
    v = None if latent else torch.where(keep[..., None, None], v, math.nan)
    return torch.randn(len(lengths), heads, dk, generator=g).to(dtype), k, v, hidden, whole, prefix_table[:len(prefixes)]


def want64(case, lengths, requests, dv, block, scale):
    q, k, v, _, whole, _ = case
    out, lse, tol, ltol = pu.attention64(q, k, v, dv, whole, lengths, requests, block, scale)
    # the part behind the prefix is rounded once more (as much again as the probabilities' rounding, of which tol counts
    # one); the two logarithms and exponentials add a few steps of fp32 of their arguments
    size = lse.abs().clamp(max=1e30)
    room = torch.where(size < 1e30, size, 0.0)
    return out, lse, tol * (2 + 2.0 ** -6 + room[..., None] * 2.0 ** -9), ltol + 2.0 ** -20 * (1 + room)


READ_ALONE = 520e6  # bytes, up to which every row reads the prefix for itself: of the prefix's table's width, the only bound that the host knows


def widened(table, rows, kv, dims, block):
    """The prefixes' table with columns that no one uses, so that even few rows share what they begin with."""
    columns = max(table.shape[1], int(READ_ALONE / (2 * rows * kv * dims * block)) + 2)
    wide = torch.full((table.shape[0], columns), -7, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


def tables(q, k, v, dv, prefix_table, block):
    """Both ways through the call."""
    yield prefix_table
    if prefix_table.shape[0]:
        yield widened(prefix_table, q.shape[0], k.shape[2], k.shape[3] + (0 if v is None else dv), block)


def check(dec, case, prefixes, prefix_of, lengths, requests, dv, block, scale=None, allowed=0, **kw):
    q, k, v, hidden, whole, prefix_table = case
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    want = want64(case, lengths, requests, dv, block, q.shape[2] ** -0.5 if scale is None else scale)
    for table in tables(q, k, v, dv, prefix_table, block):
        out, lse = dec.shared_attention(c(q), c(k), c(hidden), ints(lengths), ints(prefix_of), ints(prefixes), c(table), v_cache=c(v), v_dim=dv, scale=scale, return_lse=True, **kw)
        ok(dec, allowed)
        pu.check_attention(out, lse, want, q.dtype)
    return out, lse


HEADS = [(32, 8, 128, 128, False), (8, 8, 64, 64, False), (6, 1, 128, 64, False), (24, 2, 72, 40, False), (16, 1, 576, 512, True), (128, 1, 576, 512, True),
         (8, 2, 256, 256, False), (40, 1, 64, 128, False), (70, 1, 128, 128, False), (3, 3, 8, 8, False)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads, kv, dk, dv, latent", HEADS)
@pytest.mark.parametrize("block", [16, 33])
def test_one_prefix(dec, dtype, heads, kv, dk, dv, latent, block):
    prefix_of = [0] * 11
    lengths = [300 + x for x in (0, 1, 2, 40, 129, 15, 16, 17, 250, 5, 6)]
    case = make(1, [300], prefix_of, lengths, list(range(11)), heads, kv, dk, dv, latent, dtype, block)
    check(dec, case, [300], prefix_of, lengths, list(range(11)), dv, block)


@pytest.mark.parametrize("heads, kv, dk, dv, latent", HEADS[:7])
def test_several_prefixes_of_many_lengths(dec, heads, kv, dk, dv, latent):
    # runs of one row and of many, requests with none, prefixes of no whole page, of nothing, and longer than a request
    prefixes = [640, 15, 0, 100, 1000, 16]
    prefix_of = [0] * 3 + [-1] + [0] + [1] * 2 + [2] + [3] * 20 + [4] * 2 + [5, -9, 4, 4, 0]
    lengths = [640, 700, 641, 50, 639, 15, 20, 3] + [100 + 3 * i for i in range(20)] + [1000, 1500, 16, 0, 800, 1002, 900]
    requests = list(range(len(lengths)))
    case = make(2, prefixes, prefix_of, lengths, requests, heads, kv, dk, dv, latent, torch.bfloat16, 16)
    check(dec, case, prefixes, prefix_of, lengths, requests, dv, 16)


@pytest.mark.parametrize("next_n", [2, 3, 7])
@pytest.mark.parametrize("latent", [False, True])
def test_drafted_tokens(dec, next_n, latent):
    dk, dv, kv, heads = (576, 512, 1, 16) if latent else (128, 128, 2, 8)
    prefix_of = [0, 0, 0, -1, 1, 1, 0]
    base = [256, 300, 400, 30, 128, 1000, 250]  # the last one's first rows see less than the prefix: nothing of it is shared
    lengths = [b + j for b in base for j in range(next_n)]
    requests = [r // next_n for r in range(len(lengths))]
    case = make(3, [256, 128], prefix_of, lengths, requests, heads, kv, dk, dv, latent, torch.float16, 32)
    check(dec, case, [256, 128], prefix_of, lengths, requests, dv, 32, next_n=next_n)
    # the same rows with their requests given one by one, of which each decides for itself
    by_row = make(3, [256, 128], prefix_of[:6] + [-1], lengths, requests, heads, kv, dk, dv, latent, torch.float16, 32)
    check(dec, by_row, [256, 128], prefix_of[:6] + [-1], lengths, requests, dv, 32, row_request=ints(requests))


@pytest.mark.parametrize("next_n, heads, kv, dk, dv, latent", [(5, 4, 1, 64, 64, False), (40, 32, 4, 64, 64, False), (150, 16, 1, 576, 512, True), (33, 128, 1, 576, 512, True)])
def test_many_rows_of_a_request(dec, next_n, heads, kv, dk, dv, latent):
    # pieces of prompts behind a prefix; one row of the third request sees less than its prefix, and one of the last sees nothing
    prefix_of, base = [0, 0, 0, -1, 1, 0], [100, 96, 100, 5, 64, 300]
    lengths = [b + j for b in base for j in range(next_n)]
    lengths[2 * next_n + next_n // 2], lengths[-1] = 95, 0
    requests = [r // next_n for r in range(len(lengths))]
    case = make(13, [100, 64], prefix_of, lengths, requests, heads, kv, dk, dv, latent, torch.bfloat16, 16)
    check(dec, case, [100, 64], prefix_of, lengths, requests, dv, 16, next_n=next_n)


def test_many_rows(dec):
    # more rows than are planned at a time, runs across that border, and more than one run for each prefix
    n = 2500
    prefix_of = [0] * 900 + [1] * 700 + [-1] * 3 + [2] * (n - 1603)
    prefixes = [64, 200, 130]
    lengths = [prefixes[p] + (7 * i) % 40 if p >= 0 else 9 for i, p in enumerate(prefix_of)]
    case = make(4, prefixes, prefix_of, lengths, list(range(n)), 4, 2, 64, 64, False, torch.float16, 8)
    check(dec, case, prefixes, prefix_of, lengths, list(range(n)), 64, 8)


@pytest.mark.parametrize("rows, latent", [(1, False), (2, True), (5, False), (40, False), (40, True)])
def test_long_prefix_of_few_rows(dec, rows, latent):
    dk, dv, kv, heads = (576, 512, 1, 16) if latent else (128, 128, 4, 16)
    lengths = [9000 + 100 * i for i in range(rows)]
    case = make(5, [9000], [0] * rows, lengths, list(range(rows)), heads, kv, dk, dv, latent, torch.bfloat16, 64)
    check(dec, case, [9000], [0] * rows, lengths, list(range(rows)), dv, 64)


def test_scores_far_apart(dec):
    # the largest scores in the prefix for some rows, behind it for others; all of them minus infinity in the prefix for some
    lengths, prefix_of = [200, 230, 130, 128], [0] * 4
    case = make(6, [128], prefix_of, lengths, list(range(4)), 4, 1, 64, 64, False, torch.bfloat16, 16)
    q, k, v, hidden, whole, prefix_table = case
    k[prefix_table[0].long(), :, 0, 0] = 30.0
    q[0, :, 0], q[1, :, 0] = 40.0, -40.0
    check(dec, case, [128], prefix_of, lengths, list(range(4)), 64, 16)
    k[prefix_table[0].long(), :, 0, 0] = -math.inf
    q[:, :, 0] = 1.0
    out, lse = check(dec, case, [128], prefix_of, lengths, list(range(4)), 64, 16)
    assert (lse[3] == -math.inf).all() and (out[3] == 0).all()


def test_strided_views_and_outputs(dec):
    lengths, prefix_of, requests = [100, 90, 180], [0, 0, 0], [0, 1, 2]
    case = make(7, [80], prefix_of, lengths, requests, 6, 2, 64, 48, False, torch.float16, 16)
    q, k, v, hidden, whole, prefix_table = case
    kv = torch.full((k.shape[0], 2, 16, 3, 64), math.nan).half().cuda()  # heads before tokens, keys and values in one buffer
    kk, vv = kv[:, :, :, 0].transpose(1, 2), kv[:, :, :, 2, :48].transpose(1, 2)
    kk.copy_(k.cuda())
    vv.copy_(v.cuda())
    out = torch.full((3, 12, 64), 9.0).half().cuda()
    wide_table, wide_prefix = torch.full((3, 40), -3, dtype=torch.int32, device="cuda"), torch.full((1, 20000), -3, dtype=torch.int32, device="cuda")
    wide_table[:, 5:5 + hidden.shape[1]], wide_prefix[:, 2:2 + prefix_table.shape[1]] = hidden.cuda(), prefix_table.cuda()
    lse = torch.empty(3, 6, device="cuda")
    got, got_lse = dec.shared_attention(q.cuda(), kk, wide_table[:, 5:5 + hidden.shape[1]], ints(lengths), ints(prefix_of), ints([80]), wide_prefix[:, 2:19000],
                                        v_cache=vv, out=out[:, 1::2, 8:56], lse=lse, return_lse=True)
    assert got_lse is lse
    pu.check_attention(got, lse, want64(case, lengths, requests, 48, 16, 64 ** -0.5), torch.float16)
    assert (out[:, ::2] == 9).all() and (out[:, :, :8] == 9).all() and (out[:, :, 56:] == 9).all()
    ok(dec)


def test_padding_rows_bad_prefixes_and_pages(dec):
    lengths, prefix_of = [100, 100, 100, 100], [0, 0, 5, 0]
    case = make(8, [64], [0, 0, -1, 0], lengths, [0, 1, 2, 3], 4, 1, 64, 64, False, torch.float16, 16)
    q, k, v, hidden, whole, prefix_table = case
    # a prefix that there is none of: the request is done by itself, and reported
    check(dec, case, [64], prefix_of, lengths, [0, 1, 2, 3], 64, 16, allowed=sar.TOPK_DEV_BAD_BLOCK)
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK
    for table in tables(q, k, v, 64, prefix_table, 16):
        dec.reset()
        # rows of no request, and one of a length that is cut to the table's width
        out, lse = dec.shared_attention(q.cuda(), k.cuda(), hidden.cuda(), ints([100, 77, 2 ** 31 - 1, 50]), ints([0, 0, -1, 0]), ints([64]), table.cuda(), v_cache=v.cuda(),
                                        row_request=ints([0, -1, 2, -4]), return_lse=True)
        assert (out[1::2] == 0).all() and (lse[1::2] == -math.inf).all() and dec.status() == sar.TOPK_DEV_LENGTH_CLAMPED
        dec.reset()
        # a page of the prefix outside the cache is skipped
        bad = table.clone()
        bad[0, 2] = k.shape[0]
        out, lse = dec.shared_attention(q.cuda(), k.cuda(), hidden.cuda(), ints(lengths), ints([0, 0, -1, 0]), ints([64]), bad.cuda(), v_cache=v.cuda(), return_lse=True)
        keep = torch.tensor([t for t in range(100) if not 32 <= t < 48], dtype=torch.int32)
        want = pu.attention64(q, k, v, 64, whole, lengths, [0, 1, 2, 3], 16, 64 ** -0.5, indices=keep.expand(4, -1))
        rows = [0, 1, 3]
        pu.check_attention(out[rows], lse[rows], tuple(x[rows] * (2.1 if i == 2 else 1) + (1e-5 if i == 3 else 0) for i, x in enumerate(want)), torch.float16)
        assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_no_prefixes_and_no_rows(dec):
    lengths = [30, 0, 200]
    case = make(9, [], [-1] * 3, lengths, [0, 1, 2], 4, 2, 64, 64, False, torch.bfloat16, 16)
    check(dec, case, [], [-1] * 3, lengths, [0, 1, 2], 64, 16)
    q, k, v, hidden, _, prefix_table = case
    out, lse = dec.shared_attention(q[:0].cuda(), k.cuda(), hidden[:0].cuda(), ints([]), ints([]), ints([]), prefix_table[:0].cuda(), v_cache=v.cuda(), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("wide", [False, True])
def test_the_same_every_time_on_a_stream_and_in_a_graph(dec, wide):
    n = 30
    lengths, prefix_of = [700 + 13 * i for i in range(n)], [0] * 20 + [1] * 10
    case = make(10, [700, 300], prefix_of, lengths, list(range(n)), 16, 4, 128, 128, False, torch.bfloat16, 32)
    q, k, v, _, whole, prefix_table = (x.cuda() for x in case)
    if wide:
        prefix_table = widened(prefix_table, n, 4, 256, 32)
    ln, of, pl = ints(lengths), ints(prefix_of), ints([700, 300])
    call = lambda **kw: dec.shared_attention(q, k, whole, ln, of, pl, prefix_table, v_cache=v, return_lse=True, **kw)  # noqa: E731
    first = call()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    # a captured call plans anew from what the tensors hold when it is replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, captured))
    shorter = [n - 1 if i % 3 else 0 for i, n in enumerate(lengths)]
    shorter[0] = 100
    ln.copy_(ints(shorter))
    graph.replay()
    torch.cuda.synchronize()
    want = call()
    assert all(torch.equal(a, b) for a, b in zip(want, captured)) and not torch.equal(want[0], first[0])
    assert (captured[0][3] == 0).all()
    ok(dec)


def test_as_attention_of_every_request_by_itself(dec):
    lengths, prefix_of = [2100 + 50 * i for i in range(24)], [0] * 24
    case = make(11, [2100], prefix_of, lengths, list(range(24)), 32, 8, 128, 128, False, torch.bfloat16, 64)
    q, k, v, hidden, whole, prefix_table = (x.cuda() for x in case)
    out, lse = dec.shared_attention(q, k, hidden, ints(lengths), ints(prefix_of), ints([2100]), widened(prefix_table, 24, 8, 256, 64), v_cache=v, return_lse=True)
    alone, alone_lse = dec.attention(q, k, whole, ints(lengths), v_cache=v, return_lse=True)
    # both round their probabilities and results: four half steps of bf16 of the mean |v|, which is below 2 here
    assert (out.double() - alone.double()).abs().max() <= 4 * 2.0 ** -8 * 2 and (lse - alone_lse).abs().max() <= 1e-4


# ---- runs of many columns -----------------------------------------------------------------------------------------

WIDE = [(32, 8, 128, 128), (8, 1, 64, 64), (24, 2, 72, 40), (64, 4, 128, 64), (5, 1, 8, 8), (200, 1, 64, 128), (3, 3, 104, 120), (256, 1, 16, 96)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads, kv, dk, dv", WIDE)
@pytest.mark.parametrize("rows", [17, 70, 129])
def test_many_columns(dec, dtype, heads, kv, dk, dv, rows):
    # one run, runs of which the last has a few columns, half a unit and whole ones; lengths that end inside a tile
    prefix_of = [0] * (rows - 5) + [1] * 5
    lengths = [(517 if p == 0 else 100) + (5 * i) % 33 for i, p in enumerate(prefix_of)]
    case = make(20, [517, 100], prefix_of, lengths, list(range(rows)), heads, kv, dk, dv, False, dtype, 11)
    check(dec, case, [517, 100], prefix_of, lengths, list(range(rows)), dv, 11)


@pytest.mark.parametrize("each", [3, 40, 130])
def test_many_columns_of_several_prefixes(dec, each):
    # more units than CTAs with short prefixes; runs of few and many columns in turn, so that the second half joins in and rests
    prefixes = [130, 16, 400, 128, 0, 256, 1000]
    counts = [each, 1, each, 2, 3, 1, each]
    prefix_of = [p for p, n in enumerate(counts) for _ in range(n)] + [-1] * 4
    lengths = [max(prefixes[p], 1) + 3 * i if p >= 0 else 40 for i, p in enumerate(prefix_of)]
    requests = list(range(len(lengths)))
    case = make(21, prefixes, prefix_of, lengths, requests, 32, 4, 64, 64, False, torch.bfloat16, 16)
    check(dec, case, prefixes, prefix_of, lengths, requests, 64, 16)


@pytest.mark.parametrize("heads, kv, dk, dv", [(16, 1, 128, 128), (24, 2, 72, 40)])
def test_many_columns_of_more_prefixes_than_rows_make_units(dec, heads, kv, dk, dv):
    # a prefix for every one or two rows: units in a few parts each, where one prefix for all would be a unit or two in many
    prefixes = [2500 - 190 * i for i in range(13)]
    prefix_of = [i // 2 for i in range(22)] + [11, 12, 12, 12]
    lengths = [prefixes[p] + 7 * i for i, p in enumerate(prefix_of)]
    requests = list(range(len(lengths)))
    case = make(24, prefixes, prefix_of, lengths, requests, heads, kv, dk, dv, False, torch.bfloat16, 16)
    check(dec, case, prefixes, prefix_of, lengths, requests, dv, 16)


def test_many_columns_with_scores_that_grow(dec):
    # scores that rise along the prefix, so that maxima move often, for some of the columns
    n = 40
    prefix_of, lengths = [0] * n, [1500 + i for i in range(n)]
    for dtype in (torch.float16, torch.bfloat16):
        case = make(22, [1500], prefix_of, lengths, list(range(n)), 8, 1, 64, 64, False, dtype, 20)
        q, k, v, hidden, whole, prefix_table = case
        rise = torch.arange(1500).float() / 10
        k[prefix_table[0].long(), :, 0, 0] = rise.view(75, 20).to(dtype)
        q[::2, ::3, 0], q[1::2, ::3, 0] = 8.0, -8.0
        check(dec, case, [1500], prefix_of, lengths, list(range(n)), 64, 20)
        k[prefix_table[0, :40].long(), :, 0, 1] = -math.inf
        q[:, :, 1] = q[:, :, 1].abs()
        check(dec, case, [1500], prefix_of, lengths, list(range(n)), 64, 20)


def test_many_columns_and_pages_outside_the_cache(dec):
    n = 30
    prefix_of, lengths = [0] * n, [300 + i for i in range(n)]
    case = make(23, [300], prefix_of, lengths, list(range(n)), 16, 2, 64, 64, False, torch.float16, 10)
    q, k, v, hidden, whole, prefix_table = case
    bad = prefix_table.clone()
    bad[0, 3], bad[0, 17], bad[0, 29] = -1, k.shape[0], 2 ** 31 - 1
    keep = torch.tensor([t for t in range(329) if t // 10 not in (3, 17, 29)], dtype=torch.int32)
    want = pu.attention64(q, k, v, 64, whole, lengths, list(range(n)), 10, 64 ** -0.5, indices=keep.expand(n, -1))
    for table in tables(q, k, v, 64, bad, 10):
        out, lse = dec.shared_attention(q.cuda(), k.cuda(), hidden.cuda(), ints(lengths), ints(prefix_of), ints([300]), table.cuda(), v_cache=v.cuda(), return_lse=True)
        pu.check_attention(out, lse, (want[0], want[1], want[2] * 2.1, want[3] + 1e-5), torch.float16)
        assert dec.status() == sar.TOPK_DEV_BAD_BLOCK
        dec.reset()


def test_many_columns_of_latent_and_wide_heads_and_drafted_tokens(dec):
    for heads, kv, dk, dv, latent in [(16, 1, 576, 512, True), (16, 2, 256, 128, False), (8, 2, 128, 128, False), (16, 1, 128, 64, True)]:
        prefix_of = [0] * 30
        lengths = [b + j for b in range(400, 430) for j in range(3)]
        requests = [r // 3 for r in range(90)]
        case = make(24, [400], prefix_of, lengths, requests, heads, kv, dk, dv, latent, torch.float16, 16)
        check(dec, case, [400], prefix_of, lengths, requests, dv, 16, next_n=3)
