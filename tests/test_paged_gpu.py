"""The paged calls against their definitions in 64 bits, at the sizes and masks where they can go wrong."""
import math

import numpy as np
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


# ---- the map ---------------------------------------------------------------------------------------------------

def plain_map(context, new, table, free, taken, block, max_tokens):
    table = [list(r) for r in table]
    columns = len(table[0]) if table else 1
    slots, lens, reqs, start, left = [], [], [], [], max_tokens
    for r, (c, n) in enumerate(zip(context, new)):
        c, n = max(c, 0), min(max(n, 0), left)
        left -= n
        start.append(len(slots))
        have, need = min(-(-c // block), columns), min(-(-(c + n) // block), columns)
        for col in range(have, need):
            table[r][col] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(c, c + n):
            b = table[r][p // block] if p // block < columns else -1
            slots.append(b * block + p % block if b >= 0 else -1)
            lens.append(p + 1)
            reqs.append(r)
    start.append(len(slots))
    tail = max_tokens - len(slots)
    return table, min(taken, len(free)), slots + [-1] * tail, lens + [0] * tail, reqs + [-1] * tail, start


def run_map(dec, context, new, table, free, taken, block, max_tokens, **kw):
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dev(table).reshape(len(context), -1) if len(context) else torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    tk = dev([taken])
    m = dec.kv_map(dev(context), dev(new), t, dev(free), tk, block, max_tokens, **kw)
    return t.tolist(), int(tk), m.slots.tolist(), m.row_lens.tolist(), m.row_request.tolist(), m.token_start.tolist()


MAPS = [  # requests, largest context, largest new, block, columns, free blocks, room in the lists
    (1, 0, 1, 16, 4, 10, 4), (1, 5, 0, 16, 4, 10, 0), (7, 40, 3, 16, 4, 40, 64), (64, 300, 1, 64, 6, 64, 64),
    (33, 50, 70, 1, 130, 4000, 4000), (40, 100, 50, 33, 8, 200, 3000), (2500, 30, 5, 8, 8, 9000, 20000),
    (5000, 9, 2, 4, 4, 9000, 12000), (3, 0, 9000, 16, 600, 1800, 30000), (600, 64, 200, 16, 20, 12000, 130000)]


@pytest.mark.parametrize("requests, ctx, new, block, columns, free, room", MAPS)
def test_map(dec, requests, ctx, new, block, columns, free, room):
    rng = np.random.default_rng(requests + block)
    context, fresh = rng.integers(0, ctx + 1, requests).tolist(), rng.integers(0, new + 1, requests).tolist()
    ids = rng.permutation(requests * columns + free).tolist()
    table = [[ids.pop() if c < -(-context[r] // block) else -1 for c in range(columns)] for r in range(requests)]
    args = (context, fresh, table, ids[:free], 3, block, room)
    want, got = plain_map(*args), run_map(dec, *args)
    for name, w, g in zip(("table", "taken", "slots", "row_lens", "row_request", "token_start"), want, got):
        assert w == g, name
    ok(dec)


def test_map_no_requests(dec):
    got = run_map(dec, [], [], [], [1, 2], 1, 16, 5)
    assert got[1:] == (1, [-1] * 5, [0] * 5, [-1] * 5, [0])


@pytest.mark.parametrize("what, args", [
    (sar.TOPK_DEV_BLOCKS_EXHAUSTED, ([0, 20, 3], [40, 1, 30], [[-1] * 6, [90, 91] + [-1] * 4, [92] + [-1] * 5], [5, 6, 7, 8], 1, 16, 80)),
    (sar.TOPK_DEV_TABLE_FULL, ([60, 64, 70], [10, 3, 2], [[9, 8, 7, 6], [5, 4, 3, 2], [1, 0, 10, 11]], [50, 51], 0, 16, 20)),
    (sar.TOPK_DEV_TOKENS_DROPPED, ([0, 10, 0], [20, 30, 9], [[-1] * 6, [9] + [-1] * 5, [-1] * 6], list(range(50, 70)), 2, 16, 37)),
    (sar.TOPK_DEV_TOKENS_DROPPED, ([0, 10, 0], [2 ** 31 - 1] * 3, [[-1] * 6] * 3, list(range(50, 70)), 2, 16, 21)),
    (0, ([-5, 3, 0], [2, -7, 3], [[-1] * 2, [9, -1], [-1, -1]], [50, 51, 52], 0, 4, 8))])
def test_map_limits(dec, what, args):
    assert run_map(dec, *args) == plain_map(*args)
    assert dec.status() == what


def test_map_out_of_place_and_again(dec):
    # taken_out beside taken: the call may be repeated on the same state with the same result
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rng = np.random.default_rng(3)
    context, new = rng.integers(0, 200, 700), rng.integers(0, 30, 700)
    table, free, taken, after = dev(np.full((700, 16), 70000)), dev(np.arange(9000)), dev([4]), dev([0])
    total = int(new.sum())
    first = dec.kv_map(dev(context), dev(new), table, free, taken, 16, total, taken_out=after)
    t1, a1 = table.clone(), int(after)
    for _ in range(20):
        again = dec.kv_map(dev(context), dev(new), table, free, taken, 16, total, taken_out=after)
        assert int(after) == a1 and int(taken) == 4 and torch.equal(table, t1)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


# ---- logits ----------------------------------------------------------------------------------------------------

def logits_case(seed, lengths, next_n, heads, dim, dtype, block, scaled, row_request=None, requests=None, columns=None):
    g = torch.Generator().manual_seed(seed)
    rows = len(lengths)
    req = row_request if row_request is not None else [r // next_n for r in range(rows)]
    n_req = requests or max(req) + 1
    longest = [max([int(n) for n, b in zip(lengths, req) if b == i] + [0]) for i in range(n_req)]
    table, blocks = pu.block_table(g, longest, block, columns=columns)
    q = torch.randn(rows, heads, dim, generator=g).to(dtype)
    keys = pu.poisoned(torch.randn(blocks, block, dim, generator=g).to(dtype), table, longest, block)
    w = torch.randn(rows, heads, generator=g)
    scales = 0.5 + torch.rand(blocks, block, generator=g) if scaled else None
    return q, w, keys, scales, table, req


def check_logits(dec, lengths, case, next_n, block, max_len, row_request=None):
    q, w, keys, scales, table, req = case
    want, tol = pu.logits64(q, w, keys, scales, table, lengths, req, block, max_len)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    out = torch.full((len(lengths), max_len), 7.25, device="cuda")
    got = dec.index_logits(c(q), c(w), c(keys), c(table), torch.tensor(lengths, dtype=torch.int32, device="cuda"), key_scales=c(scales), next_n=next_n,
                           row_request=None if row_request is None else torch.tensor(row_request, dtype=torch.int32, device="cuda"), out=out).cpu().double()
    past = want.isnan()
    assert (got[past] == 7.25).all(), "written past a row's length"
    far = (got - want).abs()[~past]
    assert (far <= tol[~past]).all(), f"{float((far / tol[~past]).max()):.2f} of the bound off"


F8 = torch.float8_e4m3fn
LENGTHS = [0, 1, 2, 127, 128, 129, 0, 255, 1000, 1]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, F8])
@pytest.mark.parametrize("heads, dim, block", [(64, 128, 64), (1, 64, 16), (8, 128, 1), (24, 96, 33), (128, 128, 128), (33, 16, 7), (17, 112, 16), (96, 128, 256)])
def test_logits(dec, dtype, heads, dim, block):
    case = logits_case(1, LENGTHS, 1, heads, dim, dtype, block, scaled=dtype == F8)
    check_logits(dec, LENGTHS, case, 1, block, 1000)
    ok(dec)


@pytest.mark.parametrize("next_n", [2, 3, 5, 10])
@pytest.mark.parametrize("dtype, heads", [(torch.bfloat16, 64), (F8, 32), (torch.float16, 128), (torch.float16, 12)])
def test_logits_of_drafted_tokens(dec, next_n, dtype, heads):
    lengths = [max(0, b + j) for b in (300, 0, 126, 1500) for j in range(next_n)]
    lengths[next_n] = 0
    case = logits_case(next_n, lengths, next_n, heads, 128, dtype, 64, scaled=True)
    check_logits(dec, lengths, case, next_n, 64, 1600)
    ok(dec)


def test_logits_with_a_request_for_each_row(dec):
    req = [0] * 9 + [2] * 3 + [1] + [2] * 2 + [3, 0, 3]
    lengths = [200 + i for i in range(9)] + [0, 130, 600, 1, 128, 129, 77, 900, 2]
    case = logits_case(5, lengths, 1, 64, 128, torch.bfloat16, 16, scaled=False, row_request=req)
    check_logits(dec, lengths, case, 1, 16, 1000, row_request=req)
    ok(dec)


def test_logits_many_rows_of_one_request(dec):
    lengths, req = [1900 + i for i in range(131)], [0] * 131
    case = logits_case(6, lengths, 1, 64, 128, torch.float16, 64, scaled=False, row_request=req)
    check_logits(dec, lengths, case, 1, 64, 2100, row_request=req)


def test_logits_padding_rows_and_bad_lengths(dec):
    # a negative request sees nothing; lengths are clamped into the table's and the output's width
    req = [0, -1, 1, -1]
    lengths = [100, 50, 64, 10]
    q, w, keys, scales, table, _ = logits_case(7, [100, 64], 1, 16, 64, torch.float16, 16, False, requests=2)
    q, w = torch.randn(4, 16, 64).half(), torch.randn(4, 16)
    want, tol = pu.logits64(q, w, keys, None, table, [100, 0, 64, 0], [0, 0, 1, 0], 16, 112)
    out = torch.full((4, 112), 7.25, device="cuda")
    got = dec.index_logits(q.cuda(), w.cuda(), keys.cuda(), table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                           row_request=torch.tensor(req, dtype=torch.int32, device="cuda"), out=out).cpu().double()
    past = want.isnan()
    assert (got[past] == 7.25).all() and ((got - want).abs()[~past] <= tol[~past]).all()
    ok(dec)
    out.fill_(7.25)
    got = dec.index_logits(q.cuda(), w.cuda(), keys.cuda(), table.cuda(), torch.tensor([-3, 50, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda"),
                           row_request=torch.tensor([0, -1, 1, -1], dtype=torch.int32, device="cuda"), out=out, max_len=60).cpu()
    assert (got[0] == 7.25).all() and (got[1] == 7.25).all() and (got[3] == 7.25).all() and (got[2, 60:] == 7.25).all() and (got[2, :60] != 7.25).all()
    assert dec.status() == sar.TOPK_DEV_LENGTH_CLAMPED


def test_logits_bad_blocks_score_the_lowest(dec):
    q, w, keys, scales, table, req = logits_case(8, [300], 1, 16, 64, torch.bfloat16, 16, False)
    table[0, 3], table[0, 7] = -1, keys.shape[0]
    got = dec.index_logits(q.cuda(), w.cuda(), keys.cuda(), table.cuda(), torch.tensor([300], dtype=torch.int32, device="cuda"), max_len=300).cpu()
    low = torch.zeros(300, dtype=torch.bool)
    low[48:64] = low[112:128] = True
    assert (got[0, low] == -math.inf).all() and got[0, ~low].isfinite().all()
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_logits_propagate_infinities_and_nan(dec):
    q, w = torch.ones(1, 2, 64).half(), torch.ones(1, 2)
    keys = torch.zeros(1, 16, 64).half()
    keys[0, 1, 5], keys[0, 2, 5], keys[0, 3, 5] = math.inf, -math.inf, math.nan
    got = dec.index_logits(q.cuda(), w.cuda(), keys.cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda"), max_len=5).cpu()[0]
    assert got[0] == 0 and got[1] == math.inf and got[2] == 0 and got[3].isnan() and got[4] == 0


def test_logits_strided_views(dec):
    # interleaved keys and scales in one buffer, a slice of the queries, a wider output
    g = torch.Generator().manual_seed(9)
    lengths = [70, 200, 15]
    table, blocks = pu.block_table(g, lengths, 32)
    big = torch.randn(blocks, 32, 3, 128, generator=g).half().cuda()
    keys = big[:, :, 1]
    q = torch.randn(3, 40, 256, generator=g).half().cuda()[:, ::2, 128:]
    w = torch.randn(3, 64, generator=g).cuda()[:, 3:23]
    both = torch.rand(blocks, 32, 5, generator=g).cuda()
    scales = both[:, :, 2]
    out = torch.full((3, 333), 7.25, device="cuda")[:, 5:255]
    got = dec.index_logits(q, w, keys, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), key_scales=scales, out=out)
    want, tol = pu.logits64(q.cpu(), w.cpu(), keys.cpu(), scales.cpu(), table, lengths, [0, 1, 2], 32, 250)
    past = want.isnan()
    assert (got.cpu()[past] == 7.25).all() and ((got.cpu().double() - want).abs()[~past] <= tol[~past]).all()


# ---- attention -------------------------------------------------------------------------------------------------

def attention_case(seed, lengths, next_n, heads, kv_heads, dk, dv, latent, dtype, block, topk=0, row_request=None):
    g = torch.Generator().manual_seed(seed)
    rows = len(lengths)
    req = row_request if row_request is not None else [r // next_n for r in range(rows)]
    n_req = max(req) + 1
    longest = [max([int(n) for n, b in zip(lengths, req) if b == i] + [0]) for i in range(n_req)]
    table, blocks = pu.block_table(g, longest, block)
    q = torch.randn(rows, heads, dk, generator=g).to(dtype)
    k = pu.poisoned(torch.randn(blocks, block, kv_heads, dk, generator=g).to(dtype), table, longest, block)
    v = None if latent else pu.poisoned(torch.randn(blocks, block, kv_heads, dv, generator=g).to(dtype), table, longest, block)
    indices = None
    if topk:
        indices = torch.full((rows, topk), -1, dtype=torch.int32)
        for r, n in enumerate(lengths):
            pick = torch.randperm(int(n), generator=g)[:topk].int()
            indices[r, :len(pick)] = pick
    return q, k, v, table, req, indices


def check_attention(dec, lengths, case, next_n, dv, block, row_request=None, scale=None, allowed=0):
    q, k, v, table, req, indices = case
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want = pu.attention64(q, k, v, dv, table, [max(0, min(int(n), table.shape[1] * block)) for n in lengths], req, block, scale, indices)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = dec.attention(c(q), c(k), c(table), i32(lengths), v_cache=c(v), v_dim=dv, indices=c(indices), scale=scale, next_n=next_n,
                             row_request=i32(row_request), return_lse=True)
    pu.check_attention(out, lse, want, q.dtype)
    ok(dec, allowed)
    return out, lse


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads, topk, block", [(16, 0, 64), (128, 0, 64), (64, 0, 1), (1, 0, 33), (128, 512, 64), (16, 130, 16), (40, 1, 7), (96, 700, 128)])
def test_latent(dec, dtype, heads, topk, block):
    case = attention_case(heads + topk, LENGTHS, 1, heads, 1, 576, 512, True, dtype, block, topk)
    check_attention(dec, LENGTHS, case, 1, 512, block)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads, kv_heads, dk, dv", [(32, 4, 128, 128), (8, 8, 64, 64), (8, 2, 256, 256), (6, 2, 80, 96), (64, 1, 192, 128), (71, 1, 64, 64),
                                                     (24, 3, 8, 8), (48, 4, 128, 64), (256, 2, 128, 128), (12, 4, 512, 512), (5, 1, 576, 256), (64, 1, 576, 512), (40, 1, 520, 320)])
def test_grouped(dec, dtype, heads, kv_heads, dk, dv):
    case = attention_case(heads + dk, LENGTHS, 1, heads, kv_heads, dk, dv, False, dtype, 16)
    check_attention(dec, LENGTHS, case, 1, dv, 16)


@pytest.mark.parametrize("dk, dv", [(64, 64), (320, 256), (128, 128), (192, 64), (512, 512), (576, 8), (72, 40), (448, 384)])
def test_other_latent_sizes(dec, dk, dv):
    lengths = [3, 700, 128, 0]
    check_attention(dec, lengths, attention_case(dk, lengths, 1, 20, 1, dk, dv, True, torch.bfloat16, 32), 1, dv, 32)
    lengths = [300, 1]
    check_attention(dec, lengths, attention_case(dv, lengths, 1, 6, 3, dk, dv, True, torch.float16, 32, topk=77), 1, dv, 32)


@pytest.mark.parametrize("next_n", [2, 3, 4, 7])
@pytest.mark.parametrize("heads, kv_heads, dk, dv, latent, topk", [(16, 1, 576, 512, True, 0), (16, 1, 576, 512, True, 200), (128, 1, 576, 512, True, 0), (32, 8, 128, 128, False, 0), (8, 2, 64, 64, False, 100)])
def test_drafted_tokens(dec, next_n, heads, kv_heads, dk, dv, latent, topk):
    lengths = [b + j for b in (300, 0, 127, 2000) for j in range(next_n)]
    lengths[next_n] = 0
    case = attention_case(next_n, lengths, next_n, heads, kv_heads, dk, dv, latent, torch.bfloat16, 64, topk)
    check_attention(dec, lengths, case, next_n, dv, 64)


def test_more_columns_than_are_packed(dec):
    # 3 rows of 512 heads over one key-value head: each row by itself, in eight blocks of 64 columns
    lengths = [200, 201, 202, 40, 41, 42]
    case = attention_case(26, lengths, 3, 512, 1, 64, 64, False, torch.float16, 16)
    check_attention(dec, lengths, case, 3, 64, 16)


@pytest.mark.parametrize("block", [8, 16, 24, 32, 48, 64, 128, 192])
def test_logits_over_pages_of_any_size(dec, block):
    lengths = [700, 129, 300, 1]
    for dtype in (torch.bfloat16, F8):
        case = logits_case(block, lengths, 1, 64, 128, dtype, block, scaled=True)
        check_logits(dec, lengths, case, 1, block, 700)
    ok(dec)


def test_a_request_for_each_row(dec):
    req = [0] * 40 + [2] * 3 + [1] + [3, 0, 3]
    lengths = [200 + i for i in range(40)] + [0, 130, 600, 1, 77, 900, 2]
    for topk in (0, 150):
        case = attention_case(11, lengths, 1, 32, 1, 576, 512, True, torch.bfloat16, 16, topk, row_request=req)
        check_attention(dec, lengths, case, 1, 512, 16, row_request=req)


@pytest.mark.parametrize("lengths", [[20000], [1, 30000, 5, 129], [9000] * 3 + [0] * 4 + [16384], list(range(0, 5200, 13))])
@pytest.mark.parametrize("latent", [True, False])
def test_long_and_ragged(dec, lengths, latent):
    # the work is split over the length: few rows, one long row among short ones, many rows
    args = (16, 1, 576, 512) if latent else (16, 4, 128, 128)
    case = attention_case(12, lengths, 1, *args, latent, torch.bfloat16, 64)
    check_attention(dec, lengths, case, 1, args[3], 64)


@pytest.mark.parametrize("rows, heads, topk", [(1, 128, 2048), (2, 16, 2048), (37, 128, 300), (153, 64, 129), (200, 8, 512)])
def test_selected_split(dec, rows, heads, topk):
    lengths = [3000 - 7 * r for r in range(rows)]
    case = attention_case(13, lengths, 1, heads, 1, 576, 512, True, torch.float16, 64, topk)
    check_attention(dec, lengths, case, 1, 512, 64)


def test_index_lists_with_gaps_repeats_and_strangers(dec):
    lengths = [500, 40, 3, 900]
    case = list(attention_case(14, lengths, 1, 16, 1, 576, 512, True, torch.bfloat16, 64, 256))
    idx = case[5]
    idx[0, ::3] = -1
    idx[0, 200] = 2 ** 31 - 1
    idx[0, 201] = 500
    idx[1, :] = -1
    idx[2, :] = 2
    idx[3, 17] = -2 ** 31
    check_attention(dec, lengths, case, 1, 512, 64)


def test_selection_feeds_attention(dec):
    # topk_ragged's own output, -1 padding and all
    lengths = [5, 700, 0, 64]
    case = list(attention_case(15, lengths, 1, 16, 1, 576, 512, True, torch.bfloat16, 64))
    sel = sar.Selector(0)
    x = torch.randn(4, 704, device="cuda")
    idx = sel(x, torch.tensor(lengths, dtype=torch.int32, device="cuda"), 64)
    case[5] = idx.cpu()
    check_attention(dec, lengths, case, 1, 512, 64)


def test_scores_of_minus_infinity_and_large_scores(dec):
    lengths = [200, 130, 90]
    q, k, v, table, req, _ = attention_case(16, lengths, 1, 4, 1, 64, 64, False, torch.bfloat16, 16)
    q = q.abs() + 0.1
    b, o = pu.tokens(table, 0, torch.arange(0, 200, 3), 16)
    k[b, o, 0, 5] = -math.inf  # some tokens of row 0
    b, o = pu.tokens(table, 1, torch.arange(130), 16)
    k[b, o, 0, 7] = -math.inf  # every token of row 1: it sees nothing
    b, o = pu.tokens(table, 2, torch.arange(90), 16)
    k[b, o] = (k[b, o].float() * torch.linspace(0, 30, 90)[:, None, None]).to(k.dtype)  # rising scores: the maximum keeps moving
    check_attention(dec, lengths, (q, k, v, table, req, None), 1, 64, 16)


def test_nan_in_a_seen_token_shows(dec):
    lengths = [200, 200]
    q, k, v, table, req, _ = attention_case(17, lengths, 1, 4, 1, 128, 128, False, torch.float16, 16)
    b, o = pu.tokens(table, 1, torch.tensor([77]), 16)
    k[b, o, 0, 3] = math.nan
    out = dec.attention(q.cuda(), k.cuda(), table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), v_cache=v.cuda())
    assert out[0].isfinite().all() and out[1].isnan().all()


@pytest.mark.parametrize("heads, kv_heads, dk, dv, latent, times", [(16, 1, 576, 512, True, 1), (8, 2, 128, 128, False, 1), (128, 1, 576, 512, True, 1),
                                                                    (16, 1, 576, 512, True, 30), (4, 2, 72, 136, False, 60), (32, 1, 128, 256, False, 30),
                                                                    (40, 1, 576, 512, False, 1), (40, 1, 448, 392, False, 20), (64, 2, 384, 512, False, 1)])
def test_tokens_of_later_rows_only(dec, heads, kv_heads, dk, dv, latent, times):
    # what a request's last row alone sees shows there, whatever it is, and in no other row
    next_n, last = 3, [300, 128, 3, 2000, 129] * times
    lengths = [max(0, n + j - 2 if i % 5 != 3 else (700, 0, n)[j]) for i, n in enumerate(last) for j in range(next_n)]
    q, k, v, table, req, _ = attention_case(24, lengths, next_n, heads, kv_heads, dk, dv, latent, torch.bfloat16, 64)
    for i, n in enumerate(last):
        b, o = pu.tokens(table, i, torch.tensor([n - 1]), 64)
        (k if latent else v)[b, o, 0, 5] = (math.nan, math.inf, -math.inf)[i % 3]
    want = pu.attention64(q, k, v, dv, table, lengths, req, 64, dk ** -0.5)
    i32 = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = dec.attention(q.cuda(), k.cuda(), table.cuda(), i32, v_cache=None if v is None else v.cuda(), v_dim=dv, next_n=next_n, return_lse=True)
    ok(dec)
    early = torch.tensor([r for r in range(len(lengths)) if r % next_n != next_n - 1])
    pu.check_attention(out[early.cuda()], lse[early.cuda()], [x[early] for x in want], torch.bfloat16)
    # where the token's weight is not zero (a score of minus infinity makes it so)
    late, group = out[next_n - 1::next_n].cpu(), heads // kv_heads
    shown = want[1][next_n - 1::next_n, :group].isfinite().logical_not() if latent else torch.ones(len(last), group, dtype=torch.bool)
    assert shown.any(1).all() and late[:, :group, 5][shown].isfinite().logical_not().all()
    if not latent:
        late[:, :group, 5] = 0
        assert late.isfinite().all()


@pytest.mark.parametrize("dk, dv", [(384, 512), (576, 512), (512, 384), (448, 392)])
def test_values_that_fill_the_ring(dec, dk, dv):
    # 64 query heads' tiles leave room for as few pieces of the cache as a tile's values have; several tiles a CTA
    lengths = [300 + 7 * i for i in range(100)]
    case = attention_case(dk, lengths, 1, 64, 1, dk, dv, False, torch.bfloat16, 64)
    check_attention(dec, lengths, case, 1, dv, 64)


def test_rising_scores_over_many_tiles(dec):
    # each tile's maximum is far above the last one's: sums have to be scaled down on the way
    lengths = [1500, 1400]
    for dtype in (torch.float16, torch.bfloat16):
        q, k, v, table, req, _ = attention_case(18, lengths, 1, 16, 1, 576, 512, True, dtype, 64)
        for r, n in enumerate(lengths):
            b, o = pu.tokens(table, r, torch.arange(n), 64)
            k[b, o] = (k[b, o].float() * torch.linspace(0.05, 4, n)[:, None, None]).to(dtype)
        check_attention(dec, lengths, (q, k, v, table, req, None), 1, 512, 64, scale=0.2)


def test_clamped_lengths_and_padding_rows(dec):
    lengths = [300, 64]
    q, k, v, table, req, _ = attention_case(19, lengths, 1, 8, 2, 64, 64, False, torch.float16, 16)
    full = table.shape[1] * 16
    q4 = torch.randn(5, 8, 64).half()
    rr = [0, -1, 1, 0, 7]
    given = [300, 40, 64, -9, 30]
    want = pu.attention64(q4, k, v, 64, table, [300, 0, 64, 0, 0], [0, 0, 1, 0, 0], 16, 0.125)
    out, lse = dec.attention(q4.cuda(), k.cuda(), table.cuda(), torch.tensor(given, dtype=torch.int32, device="cuda"), v_cache=v.cuda(),
                             row_request=torch.tensor(rr, dtype=torch.int32, device="cuda"), return_lse=True)
    pu.check_attention(out, lse, want, torch.float16)
    assert dec.status() == sar.TOPK_DEV_LENGTH_CLAMPED | sar.TOPK_DEV_BAD_BLOCK
    assert full >= 300


def test_bad_blocks_are_skipped(dec):
    lengths = [300]
    q, k, v, table, req, _ = attention_case(20, lengths, 1, 8, 1, 64, 64, False, torch.float16, 16)
    bad = table.clone()
    bad[0, 2], bad[0, 5] = -1, k.shape[0] + 5
    keep = torch.tensor([[t for t in range(300) if t // 16 not in (2, 5)]], dtype=torch.int32)
    want = pu.attention64(q, k, v, 64, table, lengths, req, 16, 0.125, keep)
    out, lse = dec.attention(q.cuda(), k.cuda(), bad.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), v_cache=v.cuda(), return_lse=True)
    pu.check_attention(out, lse, want, torch.float16)
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_strided_views(dec):
    g = torch.Generator().manual_seed(21)
    lengths = [70, 200, 15]
    table, blocks = pu.block_table(g, lengths, 32)
    wide = torch.full((3, 11), -1, dtype=torch.int32)
    wide[:, 2:2 + table.shape[1]] = table
    kv = torch.randn(blocks, 2, 4, 32, 144, generator=g).bfloat16()  # keys and values beside each other, heads before tokens
    k, v = kv[:, 0].transpose(1, 2)[..., 8:136], kv[:, 1].transpose(1, 2)[..., :64]
    q = torch.randn(8, 3, 160, generator=g).bfloat16().transpose(0, 1)[..., 16:144]
    want = pu.attention64(q, k, v, 64, table, lengths, [0, 1, 2], 32, 0.1)
    kvc, qc = kv.cuda(), torch.empty(8, 3, 160, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., 16:144]
    qc.copy_(q)
    out = torch.full((3, 20, 72), 7.25, dtype=torch.bfloat16, device="cuda")
    view = out[:, 2:18:2, 8:]
    lse = torch.empty(3, 8, device="cuda")
    dec.attention(qc, kvc[:, 0].transpose(1, 2)[..., 8:136], wide.cuda()[:, 2:2 + table.shape[1]], torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                  v_cache=kvc[:, 1].transpose(1, 2)[..., :64], scale=0.1, out=view, lse=lse)
    pu.check_attention(view, lse, want, torch.bfloat16)
    out[:, 2:18:2, 8:] = 7.25
    assert (out == 7.25).all(), "written outside the view"


def test_offsets_past_32_bits(dec):
    # 5.2 GB of cache, the tokens in its last blocks
    block, blocks, dk = 64, 70000, 576
    k = torch.empty((blocks, block, 1, dk), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(22)
    lengths = [150, 64]
    table = torch.tensor([[blocks - 1, 3, blocks - 3], [blocks - 2, -1, -1]], dtype=torch.int32)
    small = torch.randn(4, block, 1, dk, generator=g).bfloat16()
    for i, b in enumerate((blocks - 1, 3, blocks - 3, blocks - 2)):
        k[b] = small[i].cuda()
    near = torch.tensor([[0, 1, 2], [3, -1, -1]], dtype=torch.int32)
    q = torch.randn(2, 16, dk, generator=g).bfloat16()
    want = pu.attention64(q, small, None, 512, near, lengths, [0, 1], block, 0.04)
    out, lse = dec.attention(q.cuda(), k, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), v_dim=512, scale=0.04, return_lse=True)
    pu.check_attention(out, lse, want, torch.bfloat16)
    w = torch.randn(2, 16, generator=g)
    keys = k.view(blocks, block, dk)[..., :128]
    lw, tol = pu.logits64(q[..., :128], w, small.view(4, block, dk)[..., :128], None, near, lengths, [0, 1], block, 192)
    got = dec.index_logits(q[..., :128].cuda(), w.cuda(), keys, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda")).cpu().double()
    past = lw.isnan()
    assert ((got - lw).abs()[~past] <= tol[~past]).all()


def test_same_answer_every_time(dec):
    # the split's join has a fixed order: repeated calls agree bit for bit
    lengths = [5000, 17, 900]
    q, k, v, table, req, _ = attention_case(23, lengths, 1, 16, 1, 576, 512, True, torch.bfloat16, 64)
    args = (q.cuda(), k.cuda(), table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    first = dec.attention(*args, v_dim=512, return_lse=True)
    for _ in range(30):
        again = dec.attention(*args, v_dim=512, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_another_stream_and_a_graph(dec):
    lengths = [3000, 17, 900, 0]
    q, k, v, table, req, _ = attention_case(24, lengths, 1, 16, 1, 576, 512, True, torch.bfloat16, 64)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    qc, kc, tc = q.cuda(), k.cuda(), table.cuda()
    want = dec.attention(qc, kc, tc, ln, v_dim=512)
    keys, w = kc[:, :, 0, :128], torch.randn(4, 16, device="cuda")
    want_l = dec.index_logits(qc[..., :128], w, keys, tc, ln, out=torch.zeros(4, 3008, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = dec.attention(qc, kc, tc, ln, v_dim=512, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    out, logits = torch.empty_like(want), torch.zeros(4, 3008, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.index_logits(qc[..., :128], w, keys, tc, ln, out=logits)
        dec.attention(qc, kc, tc, ln, v_dim=512, out=out)
    for _ in range(3):
        out.zero_()
        logits.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out) and torch.equal(want_l, logits)
    ok(dec)


def test_binding_refuses(dec):
    q, k = torch.zeros(2, 16, 64, device="cuda").half(), torch.zeros(3, 16, 1, 64, device="cuda").half()
    t, ln = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q.bfloat16()), dict(k_cache=k.cpu()), dict(lengths=ln.long()), dict(lengths=ln[:1]), dict(block_table=t.long()),
                dict(v_dim=None), dict(indices=t.long()), dict(out=torch.zeros(2, 16, 32, device="cuda").half()), dict(row_request=ln[:1])):
        with pytest.raises(ValueError):
            dec.attention(**{**dict(q=q, k_cache=k, block_table=t, lengths=ln, v_dim=64), **bad})
    with pytest.raises(sar.TopkError):
        dec.attention(q, k, t, ln, v_dim=72)
    with pytest.raises(ValueError):
        dec.index_logits(q, torch.zeros(2, 15, device="cuda"), k[:, :, 0], t, ln)


# ---- together ----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [dict(), dict(requests=1, prompt=40, topk=64, block=16, heads=128), dict(requests=9, prompt=300, topk=1, block=5, heads=40),
                                dict(requests=3, prompt=2500, topk=2048, heads=64)])
def test_example_of_sparse_decoding(dec, kw):
    # map, logits, selection and attention, each call on the last one's output; bf16 outputs below 8, so half a unit in
    # the last place of the largest (2^-6), as much for the probabilities' rounding, and the same again
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_decode.py")
    spec = importlib.util.spec_from_file_location("sparse_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.run(**kw) < 4 * 2.0 ** -6
