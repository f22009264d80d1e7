"""The paged calls where they went wrong once."""
import pytest
import torch

import sparse_attention_row_gb300 as sar
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


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_map_reports_tokens_on_a_page_that_an_earlier_step_did_not_get(dec):
    # the free list ends within request 0's new tokens; the next step's token falls into the page that was entered as -1
    table, free, taken = dev([[-1] * 4, [9, 8, -1, -1]]), dev([5, 6]), dev([0])
    first = dec.kv_map(dev([0, 20]), dev([40, 1]), table, free, taken, 16, 41)
    assert table.tolist() == [[5, 6, -1, -1], [9, 8, -1, -1]] and int(taken) == 2
    assert first.slots.tolist() == list(range(80, 112)) + [-1] * 8 + [8 * 16 + 4]
    assert dec.status() == sar.TOPK_DEV_BLOCKS_EXHAUSTED
    dec.reset()
    second = dec.kv_map(dev([40, 21]), dev([1, 1]), table, free, taken, 16, 2)
    assert second.slots.tolist() == [-1, 8 * 16 + 5]
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_map_reports_a_negative_block_on_the_free_list(dec):
    table = dev([[-1] * 2])
    m = dec.kv_map(dev([0]), dev([20]), table, dev([3, -7]), dev([0]), 16, 20)
    assert m.slots.tolist() == list(range(48, 64)) + [-1] * 4 and table.tolist() == [[3, -7]]
    assert dec.status() == sar.TOPK_DEV_BAD_BLOCK


def test_a_new_decoder_is_ready_on_another_stream(dec):
    # its workspace comes dirty from the allocator, and the stream that it is made on has work to do; the call is made on
    # another stream at once
    requests, each, block = 64, 100, 16
    context, new, table = dev([0] * requests), dev([each] * requests), dev([[-1] * 7] * requests)
    free, taken, after, side = dev(list(range(7 * requests))), dev([0]), dev([0]), torch.cuda.Stream()
    junk = torch.full((dec.nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(200_000_000)
    fresh = sar.PagedDecoder(0)
    fresh.kv_map(context, new, table, free, taken, block, requests * each, taken_out=after, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert int(after) == 7 * requests
    assert fresh.status() == 0


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_finite_scores_far_below_zero_after_scores_of_minus_infinity(dec, dtype, listed):
    # a row's first 128 tokens score -inf, the others all the same: a finite number, for bf16 far below -1e30. 160 rows, so
    # that both tiles of a row are one run's, of 16 heads, so that no column is left over. Probabilities are one; their sums
    # and the values' are exact but for the last steps: the mean of 64 values of half a unit, three roundings of the
    # log-sum and two of its constants.
    heads, dk, tokens, block, scale = 16, 64, 192, 64, 0.125
    q = torch.full((160, heads, dk), 2.0 ** (60 if dtype == torch.bfloat16 else 6), dtype=dtype)
    k = torch.zeros(3, block, 1, dk, dtype=dtype)
    k[:2, :, 0, 5] = -float("inf")
    k[2, :, 0, 7] = -2.0 ** (50 if dtype == torch.bfloat16 else 8)
    v = torch.randn(3, block, 1, dk, generator=torch.Generator().manual_seed(1)).to(dtype)
    table = torch.arange(3, dtype=torch.int32).repeat(160, 1)
    indices = torch.arange(tokens, dtype=torch.int32).repeat(160, 1) if listed else None
    score = scale * float(q[0, 0, 0]) * float(k[2, 0, 0, 7])
    out, lse = dec.attention(q.cuda(), k.cuda(), table.cuda(), dev([tokens] * 160), v_cache=v.cuda(), scale=scale, return_lse=True,
                             indices=None if indices is None else indices.cuda())
    assert dec.status() == 0
    want = v[2, :, 0].double().mean(0)
    half = 2.0 ** (-11 if dtype == torch.float16 else -8)
    room = want.abs() * half * 1.01 + v[2].double().abs().mean() * 64 * 2.0 ** -22
    assert ((out.cpu().double() - want).abs() <= room).all()
    log_sum = score + 4.1588830833596715  # ln 64
    assert ((lse.cpu().double() - log_sum).abs() <= abs(log_sum) * 2.0 ** -21).all()
