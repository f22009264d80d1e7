"""Forms of the paged calls beside the ordinary ones: without dependent launch, on two streams at once, other layouts."""
import os
import subprocess
import sys

import pytest
import torch

import sparse_attention_row_gb300 as sar
from tests import paged_util as pu
from tests import test_paged_gpu as base
from tests.gpu_util import require_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dec():
    require_cuda()
    return sar.PagedDecoder(0)


@pytest.fixture(autouse=True)
def _clear(request):
    yield
    if "dec" in request.fixturenames:
        request.getfixturevalue("dec").reset()


@pytest.mark.parametrize("switch", ["1", "2"])
def test_example_with_and_without_dependent_launch(switch):
    # the switch is read once in a process: map, logits, selection and attention in one of its own
    require_cuda()
    code = ("import importlib.util as u; s = u.spec_from_file_location('e', 'examples/sparse_decode.py'); m = u.module_from_spec(s); "
            "s.loader.exec_module(m); w = m.run(requests=3, prompt=400, topk=128); assert w < 4 * 2.0 ** -6, w")
    env = dict(os.environ, LIBTOPK_DEPENDENT_LAUNCH=switch)
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, done.stderr


def test_a_workspace_that_is_too_small_is_refused(dec):
    q, k = torch.zeros(1, 16, 64, device="cuda").half(), torch.zeros(1, 16, 1, 64, device="cuda").half()
    table, lengths, out = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"), torch.full_like(q, 7.25)
    rows = sar.TopkPagedRows(num_rows=1, next_n=1, block_size=16, num_requests=1, num_blocks=1, lengths=lengths.data_ptr(),
                             block_table=table.data_ptr(), table_stride=1, max_blocks=1)
    args = sar.TopkAttentionArgs(rows=rows, dtype=sar.TOPK_DTYPE_F16, heads=16, kv_heads=1, dk=64, dv=64, scale=0.125, q=q.data_ptr(), q_row_stride=1024,
                                 q_head_stride=64, k=k.data_ptr(), k_block_stride=1024, k_token_stride=64, k_head_stride=64, out=out.data_ptr(),
                                 out_row_stride=1024, out_head_stride=64, workspace=dec.workspace.data_ptr(), workspace_bytes=dec.nbytes - 1)
    assert sar.topk_paged_attention(args) == sar.TOPK_ERR_WORKSPACE_TOO_SMALL
    torch.cuda.synchronize()
    assert (out == 7.25).all()
    args.workspace_bytes = dec.nbytes
    assert sar.topk_paged_attention(args) == sar.TOPK_OK
    torch.cuda.synchronize()
    assert (out == 0).all() and dec.status() == 0


@pytest.mark.parametrize("heads, kv_heads, dk, dv", [(32, 4, 128, 128), (5, 1, 64, 128), (96, 2, 256, 64)])
@pytest.mark.parametrize("topk", [0, 100])
def test_grouped_heads_with_a_request_for_each_row(dec, heads, kv_heads, dk, dv, topk):
    # rows of mixed requests, one that sees nothing, padding rows among them
    req = [2, 2, 0, 0, 0, 3, 1, 0, 2, 3, 3]
    lengths = [300, 301, 128, 129, 0, 5, 700, 40, 1, 6, 7]
    case = base.attention_case(31, lengths, 1, heads, kv_heads, dk, dv, False, torch.float16, 16, topk, row_request=req)
    q, k, v, table, _, indices = case
    pads = [1, 5, 10]  # before these rows
    given_req, given_len, at = [], [], []
    for r in range(len(req)):
        if r in pads:
            given_req.append(-1)
            given_len.append(99)
        at.append(len(given_req))
        given_req.append(req[r])
        given_len.append(lengths[r])
    wide_q = torch.full((len(given_req), heads, dk), float("nan"), dtype=q.dtype)
    wide_q[at] = q
    wide_i = None
    if indices is not None:
        wide_i = torch.zeros((len(given_req), topk), dtype=torch.int32)
        wide_i[at] = indices
        wide_i = wide_i.cuda()
    want = pu.attention64(q, k, v, dv, table, lengths, req, 16, dk ** -0.5, indices)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = dec.attention(wide_q.cuda(), k.cuda(), table.cuda(), i32(given_len), v_cache=v.cuda(), indices=wide_i, row_request=i32(given_req), return_lse=True)
    pu.check_attention(out[at], lse[at], want, q.dtype)
    pad_rows = [r for r in range(len(given_req)) if r not in at]
    assert (out[pad_rows] == 0).all() and (lse[pad_rows] == -float("inf")).all()
    assert dec.status() == 0


def test_two_decoders_on_two_streams(dec):
    # calls that overlap, each with a workspace of its own, agree with the same calls alone
    other = sar.PagedDecoder(0)
    lengths = [3000, 17, 900, 2500, 128, 4000]
    q, k, _, table, _, _ = (x.cuda() if isinstance(x, torch.Tensor) else x for x in base.attention_case(33, lengths, 1, 16, 1, 576, 512, True, torch.bfloat16, 64))
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    keys, w, tk = k[:, :, 0, :128], torch.randn(6, 16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    free, zeros = torch.arange(6 * 48, dtype=torch.int32, device="cuda"), torch.zeros_like(ln)

    def calls(d, stream):
        t, taken = torch.zeros_like(table), torch.zeros_like(tk)
        logits = torch.zeros(6, 4032, device="cuda")
        torch.cuda.synchronize()
        made = []
        for _ in range(8):
            out, lse = d.attention(q, k, table, ln, v_dim=512, return_lse=True, stream=stream)
            d.index_logits(q[..., :128], w, keys, table, ln, out=logits, stream=stream)
            m = d.kv_map(zeros, ln, t, free, tk, 64, 12000, taken_out=taken, stream=stream)
            made.append([out, lse, logits, taken, *m])
        return made

    want = calls(dec, None)[0]
    torch.cuda.synchronize()
    want = [x.clone() for x in want]
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = calls(dec, first), calls(other, second)
    torch.cuda.synchronize()
    for made in a + b:
        for x, y in zip(made, want):
            assert torch.equal(x, y)
    assert dec.status() == 0 and other.status() == 0


@pytest.mark.parametrize("extra", [8, 24, 64, 128])
@pytest.mark.parametrize("block", [16, 20])
def test_logits_with_gaps_between_the_pages(dec, extra, block):
    # block and token strides whose common divisor is smaller than a key
    lengths, dim = [300, 77, 129], 128
    q, w, keys, _, table, req = base.logits_case(41, lengths, 1, 40, dim, torch.bfloat16, block, scaled=False)
    blocks = keys.shape[0]
    flat = torch.full((blocks * (block * dim + extra),), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = flat.view(blocks, -1)[:, :block * dim].view(blocks, block, dim)
    view.copy_(keys)
    assert view.stride(0) == block * dim + extra
    want, tol = pu.logits64(q, w, keys, None, table, lengths, req, block, 300)
    out = torch.full((3, 300), 7.25, device="cuda")
    got = dec.index_logits(q.cuda(), w.cuda(), view, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), out=out).cpu().double()
    past = want.isnan()
    assert (got[past] == 7.25).all() and ((got - want).abs()[~past] <= tol[~past]).all()
    assert dec.status() == 0
