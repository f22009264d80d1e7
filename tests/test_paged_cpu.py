"""The paged calls' argument structs and what they refuse on the host (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import sparse_attention_row_gb300 as sar
from sparse_attention_row_gb300 import build, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: validation fails before any CUDA call

STRUCTS = {"topk_paged_rows": sar.TopkPagedRows, "topk_kv_map_args": sar.TopkKvMapArgs,
           "topk_index_logits_args": sar.TopkIndexLogitsArgs, "topk_attention_args": sar.TopkAttentionArgs}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "libtopk.h"', "int main(void) {"]
    for cname, py in STRUCTS.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.check_call([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in subprocess.check_output([str(exe)], text=True).splitlines()}
    for cname, py in STRUCTS.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


@pytest.mark.parametrize("packer, struct", [(paged._MAP, sar.TopkKvMapArgs), (paged._LOGITS, sar.TopkIndexLogitsArgs), (paged._ATTENTION, sar.TopkAttentionArgs)])
def test_packed_arguments_have_the_structs_layout(packer, struct):
    def leaves(s, at=0):
        for name, kind in s._fields_:
            if issubclass(kind, ctypes.Structure):
                yield from leaves(kind, at + getattr(s, name).offset)
            else:
                yield name, kind, at + getattr(s, name).offset

    fields = list(leaves(struct))
    assert packer.size == ctypes.sizeof(struct)
    values = [float(i + 1) if kind is ctypes.c_float else i + 1 for i, (_, kind, _) in enumerate(fields)]
    data = packer.pack(*values)
    for value, (name, kind, at) in zip(values, fields):
        assert kind.from_buffer_copy(data, at).value == value, name


def test_header_constants():
    text = open(os.path.join(ROOT, "include", "libtopk.h")).read()
    for name, value in re.findall(r"#define (TOPK_DEV_\w+) (0x[0-9a-f]+)u", text):
        assert getattr(sar, name) == int(value, 16), name
    assert re.search(r"TOPK_ERR_UNSUPPORTED = 9\b", text) and sar.TOPK_ERR_UNSUPPORTED == 9
    assert f"TOPK_PAGED_WORKSPACE_BYTES {sar.TOPK_PAGED_WORKSPACE_BYTES}" in text
    assert sar.topk_status_string(9).startswith("unsupported")


def rows(**kw):
    r = dict(num_rows=4, next_n=1, block_size=16, num_requests=4, num_blocks=10, lengths=FAKE, row_request=None,
             block_table=FAKE, table_stride=8, max_blocks=8)
    r.update({k: v for k, v in kw.items() if k in r})
    return sar.TopkPagedRows(**r)


def map_args(**kw):
    a = dict(context_lens=FAKE, new_lens=FAKE, num_requests=4, block_size=16, block_table=FAKE, table_stride=8, max_blocks=8,
             free_blocks=FAKE, num_free=10, taken=FAKE, taken_out=FAKE, slots=FAKE, row_lens=FAKE, row_request=FAKE,
             token_start=FAKE, max_tokens=100, workspace=FAKE)
    a.update(kw)
    return sar.TopkKvMapArgs(**a)


def logits_args(**kw):
    a = dict(dtype=sar.TOPK_DTYPE_BF16, heads=64, dim=128, q=FAKE, q_row_stride=8192, q_head_stride=128, weights=FAKE,
             weight_row_stride=64, keys=FAKE, key_block_stride=2048, key_token_stride=128, key_scales=None, scale_block_stride=16,
             scale_token_stride=1, logits=FAKE, logits_row_stride=128, max_len=128, workspace=FAKE)
    a.update({k: v for k, v in kw.items() if k in a})
    return sar.TopkIndexLogitsArgs(rows=rows(**kw), **a)


def attention_args(**kw):
    a = dict(dtype=sar.TOPK_DTYPE_BF16, heads=16, kv_heads=1, dk=576, dv=512, scale=0.04, q=FAKE, q_row_stride=9216, q_head_stride=576,
             k=FAKE, k_block_stride=9216, k_token_stride=576, k_head_stride=576, v=None, v_block_stride=0, v_token_stride=0,
             v_head_stride=0, indices=None, index_row_stride=512, num_indices=512, out=FAKE, out_row_stride=8192,
             out_head_stride=512, lse=None, workspace=FAKE, workspace_bytes=1 << 40)
    a.update({k: v for k, v in kw.items() if k in a})
    return sar.TopkAttentionArgs(rows=rows(**kw), **a)


BAD, MIS, UNS = sar.TOPK_ERR_INVALID_ARG, sar.TOPK_ERR_MISALIGNED, sar.TOPK_ERR_UNSUPPORTED
ROW_REFUSALS = [(BAD, dict(num_rows=-1)), (BAD, dict(num_rows=1 << 31)), (BAD, dict(next_n=0)), (BAD, dict(next_n=3)),
                (BAD, dict(num_requests=3)), (BAD, dict(block_size=0)), (BAD, dict(max_blocks=0)), (BAD, dict(table_stride=7)),
                (BAD, dict(lengths=None)), (BAD, dict(block_table=None)), (MIS, dict(lengths=FAKE + 2)),
                (MIS, dict(block_table=FAKE + 1)), (BAD, dict(num_blocks=-1)), (BAD, dict(workspace=None)), (MIS, dict(workspace=FAKE + 8))]


@pytest.mark.parametrize("code, change", [
    (BAD, dict(num_requests=-1)), (BAD, dict(block_size=0)), (BAD, dict(max_blocks=0)), (BAD, dict(table_stride=7)), (BAD, dict(num_free=-1)),
    (BAD, dict(max_tokens=-1)), (BAD, dict(max_tokens=1 << 31)), (BAD, dict(context_lens=None)), (BAD, dict(taken=None)),
    (BAD, dict(free_blocks=None)), (BAD, dict(slots=None)), (BAD, dict(workspace=None)), (MIS, dict(slots=FAKE + 4)), (MIS, dict(new_lens=FAKE + 2))])
def test_map_refusals(code, change):
    assert sar.topk_kv_map(map_args(**change), 0) == code


@pytest.mark.parametrize("code, change", ROW_REFUSALS + [
    (UNS, dict(dtype=0)), (UNS, dict(dtype=4)), (UNS, dict(heads=0)), (UNS, dict(heads=129)), (UNS, dict(dim=0)), (UNS, dict(dim=136)),
    (UNS, dict(dim=12)), (UNS, dict(dim=24, dtype=3)), (BAD, dict(max_len=0)), (BAD, dict(logits_row_stride=-1)), (BAD, dict(q=None)), (BAD, dict(weights=None)),
    (BAD, dict(keys=None)), (BAD, dict(logits=None)), (MIS, dict(q=FAKE + 8)), (MIS, dict(key_token_stride=132)), (MIS, dict(key_scales=FAKE + 2))])
def test_logits_refusals(code, change):
    assert sar.topk_index_logits(logits_args(**change), 0) == code


@pytest.mark.parametrize("code, change", ROW_REFUSALS + [
    (UNS, dict(dtype=3)), (UNS, dict(dtype=0)), (BAD, dict(heads=0)), (BAD, dict(kv_heads=0)), (BAD, dict(kv_heads=3)), (UNS, dict(heads=1025)),
    (UNS, dict(dk=584)), (UNS, dict(dk=4)), (UNS, dict(dk=60)), (UNS, dict(dv=520)), (UNS, dict(dk=64, dv=128)), (UNS, dict(dv=4)), (BAD, dict(scale=0.0)),
    (BAD, dict(scale=-1.0)), (BAD, dict(scale=float("nan"))), (BAD, dict(scale=float("inf"))), (BAD, dict(indices=FAKE, num_indices=0)),
    (BAD, dict(indices=FAKE, index_row_stride=-1)), (BAD, dict(indices=FAKE, num_indices=(1 << 20) + 1)), (BAD, dict(q=None)), (BAD, dict(k=None)), (BAD, dict(out=None)), (MIS, dict(q=FAKE + 8)),
    (MIS, dict(k_token_stride=580)), (MIS, dict(out_head_stride=4)), (MIS, dict(v=FAKE + 2)), (MIS, dict(indices=FAKE + 2)), (MIS, dict(lse=FAKE + 1))])
def test_attention_refusals(code, change):
    assert sar.topk_paged_attention(attention_args(**change), 0) == code


def test_no_rows_is_no_work():
    assert sar.topk_index_logits(logits_args(num_rows=0, lengths=None, q=None), 0) == sar.TOPK_OK
    assert sar.topk_paged_attention(attention_args(num_rows=0, lengths=None, q=None), 0) == sar.TOPK_OK
