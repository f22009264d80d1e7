"""Argument structs, refusals on the host, and the sources of the calls for blocks, shared prefixes and pages (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import sparse_attention_row_gb300 as sar
from sparse_attention_row_gb300 import build, paged
from tests import test_paged_cpu as base
from tests import test_paged_source_cpu as source

FAKE, BAD, MIS, UNS = base.FAKE, base.BAD, base.MIS, base.UNS
SMALL = sar.TOPK_ERR_WORKSPACE_TOO_SMALL

STRUCTS = {"topk_block_means_args": (paged._MEANS, sar.TopkBlockMeansArgs), "topk_block_scores_args": (paged._SCORES, sar.TopkBlockScoresArgs),
           "topk_block_attention_args": (paged._BLOCKS, sar.TopkBlockAttentionArgs), "topk_shared_attention_args": (paged._SHARED, sar.TopkSharedAttentionArgs),
           "topk_page_fork_args": (paged._FORK, sar.TopkPageForkArgs), "topk_page_free_args": (paged._FREE, sar.TopkPageFreeArgs),
           "topk_page_compact_args": (paged._COMPACT, sar.TopkPageCompactArgs), "topk_page_copy_args": (paged._COPY, sar.TopkPageCopyArgs),
           "topk_page_cache": (paged._CACHE, sar.TopkPageCache), "topk_page_pool": (None, sar.TopkPagePool)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "libtopk.h"', "int main(void) {"]
    for cname, (_, py) in STRUCTS.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.check_call([cc, "-std=c99", "-I", os.path.join(base.ROOT, "include"), str(src), "-o", str(exe)])
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in subprocess.check_output([str(exe)], text=True).splitlines()}
    for cname, (_, py) in STRUCTS.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


@pytest.mark.parametrize("packer, struct", [x for x in STRUCTS.values() if x[0] is not None])
def test_packed_arguments_have_the_structs_layout(packer, struct):
    assert ctypes.sizeof(struct) - 8 < packer.size <= ctypes.sizeof(struct)  # but for padding at the end
    fields = []

    def leaves(s, at=0):
        for name, kind in s._fields_:
            if issubclass(kind, ctypes.Structure):
                leaves(kind, at + getattr(s, name).offset)
            else:
                fields.append((name, kind, at + getattr(s, name).offset))

    leaves(struct)
    values = [float(i + 1) if kind is ctypes.c_float else i + 1 for i, (_, kind, _) in enumerate(fields)]
    data = packer.pack(*values)
    for value, (name, kind, at) in zip(values, fields):
        assert kind.from_buffer_copy(data, at).value == value, name


def test_header_constants():
    text = open(os.path.join(base.ROOT, "include", "libtopk.h")).read()
    assert f"#define TOPK_MAX_PAGE_CACHES {sar.TOPK_MAX_PAGE_CACHES}\n" in text


def fill(struct, defaults, change):
    a = dict(defaults)
    a.update({k: v for k, v in change.items() if k in a})
    return struct(**a)


def means_args(**kw):
    return fill(sar.TopkBlockMeansArgs, dict(context_lens=FAKE, new_lens=FAKE, num_requests=4, block_size=16, dtype=sar.TOPK_DTYPE_BF16, block_table=FAKE, table_stride=8, max_blocks=8,
                                             num_blocks=10, kv_heads=2, dk=64, k=FAKE, k_block_stride=2048, k_token_stride=128, k_head_stride=64, means=FAKE, mean_block_stride=128,
                                             mean_head_stride=64, workspace=FAKE), kw)


def scores_args(**kw):
    rest = dict(dtype=sar.TOPK_DTYPE_BF16, heads=8, kv_heads=2, dk=64, sink_blocks=0, recent_blocks=0, q=FAKE, q_row_stride=512, q_head_stride=64, means=FAKE, mean_block_stride=128,
                mean_head_stride=64, scores=FAKE, score_row_stride=16, score_head_stride=8, max_columns=8, score_lens=FAKE, workspace=FAKE)
    return fill(sar.TopkBlockScoresArgs, dict(rows=base.rows(**kw), **rest), kw)


def blocks_args(**kw):
    return fill(sar.TopkBlockAttentionArgs, dict(attention=base.attention_args(**kw), blocks=FAKE, block_row_stride=4, block_head_stride=4, num_chosen=4), kw)


def shared_args(**kw):
    kw = dict(dict(lse=FAKE), **kw)
    return fill(sar.TopkSharedAttentionArgs, dict(attention=base.attention_args(**kw), prefix_of=FAKE, num_prefixes=2, prefix_lens=FAKE, prefix_table=FAKE, prefix_stride=4, prefix_blocks=4,
                                                  scratch=FAKE, scratch_bytes=1 << 40), kw)


def pool(**kw):
    return fill(sar.TopkPagePool, dict(block_table=FAKE, num_requests=4, table_stride=8, max_blocks=8, shares=FAKE, num_blocks=10, free_blocks=FAKE, num_free=10, taken=FAKE, workspace=FAKE), kw)


def fork_args(**kw):
    return fill(sar.TopkPageForkArgs, dict(pool=pool(**kw), parents=FAKE, children=FAKE, kept_lens=FAKE, num_forks=2, block_size=16, source=FAKE, target=FAKE), kw)


def free_args(**kw):
    return fill(sar.TopkPageFreeArgs, dict(pool=pool(**kw), requests=FAKE, num_freed=2), kw)


def compact_args(**kw):
    return fill(sar.TopkPageCompactArgs, dict(pool=pool(**kw), max_copies=4, source=FAKE, target=FAKE, block_table_out=FAKE, table_out_stride=8, shares_out=FAKE, free_blocks_out=FAKE,
                                              taken_out=FAKE, scratch=FAKE, scratch_bytes=1000), kw)


def copy_args(**kw):
    cache = fill(sar.TopkPageCache, dict(base=FAKE, num_blocks=10, block_stride=256, stride0=0, stride1=0, n0=1, n1=1, run_bytes=256), kw)
    held = ctypes.pointer(cache)
    a = fill(sar.TopkPageCopyArgs, dict(source=FAKE, target=FAKE, num_copies=4, caches=ctypes.cast(held, ctypes.c_void_p), num_caches=1, workspace=FAKE), kw)
    a.held = held
    return a


@pytest.mark.parametrize("code, change", [
    (BAD, dict(num_requests=-1)), (BAD, dict(block_size=0)), (BAD, dict(max_blocks=0)), (BAD, dict(table_stride=7)), (BAD, dict(num_blocks=-1)), (BAD, dict(kv_heads=0)), (UNS, dict(dtype=0)),
    (UNS, dict(dtype=3)), (UNS, dict(kv_heads=1025)), (UNS, dict(dk=4)), (UNS, dict(dk=60)), (UNS, dict(dk=584)), (BAD, dict(context_lens=None)), (BAD, dict(new_lens=None)),
    (BAD, dict(block_table=None)), (BAD, dict(k=None)), (BAD, dict(means=None)), (BAD, dict(workspace=None)), (MIS, dict(k=FAKE + 8)), (MIS, dict(k_token_stride=68)),
    (MIS, dict(means=FAKE + 2)), (MIS, dict(mean_head_stride=4)), (MIS, dict(context_lens=FAKE + 2)), (MIS, dict(workspace=FAKE + 8)),
    (UNS, dict(num_requests=2000, max_blocks=1 << 23, table_stride=1 << 23))])
def test_means_refusals(code, change):
    assert sar.topk_block_means(means_args(**change), 0) == code


@pytest.mark.parametrize("code, change", base.ROW_REFUSALS + [
    (UNS, dict(dtype=0)), (UNS, dict(dtype=3)), (BAD, dict(heads=0)), (BAD, dict(kv_heads=0)), (BAD, dict(kv_heads=3)), (UNS, dict(heads=1026)), (UNS, dict(dk=4)), (UNS, dict(dk=584)),
    (BAD, dict(sink_blocks=-1)), (BAD, dict(recent_blocks=-1)), (BAD, dict(max_columns=0)), (BAD, dict(score_row_stride=-1)), (BAD, dict(score_head_stride=-1)), (BAD, dict(q=None)),
    (BAD, dict(means=None)), (BAD, dict(scores=None)), (BAD, dict(score_lens=None)), (MIS, dict(q=FAKE + 8)), (MIS, dict(q_head_stride=4)), (MIS, dict(mean_block_stride=4)),
    (MIS, dict(scores=FAKE + 2)), (MIS, dict(score_lens=FAKE + 1))])
def test_scores_refusals(code, change):
    assert sar.topk_block_scores(scores_args(**change), 0) == code


ATTENTION = [x for x in base.test_attention_refusals.pytestmark[0].args[1] if x[1].get("indices") is None]


@pytest.mark.parametrize("code, change", ATTENTION + [
    (BAD, dict(indices=FAKE)), (BAD, dict(num_chosen=0)), (BAD, dict(num_chosen=1 << 26)), (BAD, dict(block_row_stride=-1)), (BAD, dict(block_head_stride=-1)), (BAD, dict(blocks=None)),
    (MIS, dict(blocks=FAKE + 2))])
def test_block_attention_refusals(code, change):
    assert sar.topk_block_attention(blocks_args(**change), 0) == code


@pytest.mark.parametrize("code, change", ATTENTION + [
    (BAD, dict(indices=FAKE)), (BAD, dict(lse=None)), (BAD, dict(prefix_of=None)), (BAD, dict(prefix_lens=None)), (BAD, dict(prefix_table=None)), (BAD, dict(num_prefixes=-1)),
    (BAD, dict(num_prefixes=1 << 31)), (BAD, dict(prefix_blocks=0)), (BAD, dict(prefix_stride=3)), (BAD, dict(scratch=None)), (MIS, dict(scratch=FAKE + 8)), (MIS, dict(prefix_of=FAKE + 2)),
    (MIS, dict(prefix_lens=FAKE + 1)), (MIS, dict(prefix_table=FAKE + 2))])
def test_shared_attention_refusals(code, change):
    assert sar.topk_shared_attention(shared_args(**change), 0) == code


POOL = [(BAD, dict(num_requests=-1)), (BAD, dict(max_blocks=0)), (BAD, dict(table_stride=7)), (BAD, dict(num_blocks=-1)), (BAD, dict(num_free=-1)), (BAD, dict(num_requests=1 << 20, max_blocks=1 << 11, table_stride=1 << 11)),
        (BAD, dict(block_table=None)), (BAD, dict(shares=None)), (BAD, dict(free_blocks=None)), (BAD, dict(taken=None)), (BAD, dict(workspace=None)), (MIS, dict(block_table=FAKE + 2)),
        (MIS, dict(shares=FAKE + 1)), (MIS, dict(free_blocks=FAKE + 2)), (MIS, dict(taken=FAKE + 2)), (MIS, dict(workspace=FAKE + 8))]


@pytest.mark.parametrize("code, change", POOL + [
    (BAD, dict(num_forks=-1)), (BAD, dict(block_size=0)), (BAD, dict(parents=None)), (BAD, dict(children=None)), (BAD, dict(kept_lens=None)), (BAD, dict(source=None)), (BAD, dict(target=None)),
    (MIS, dict(parents=FAKE + 2)), (MIS, dict(target=FAKE + 1))])
def test_fork_refusals(code, change):
    assert sar.topk_page_fork(fork_args(**change), 0) == code


@pytest.mark.parametrize("code, change", POOL + [
    (BAD, dict(num_freed=-1)), (BAD, dict(num_freed=(1 << 20) + 1)), (BAD, dict(num_freed=1 << 18, max_blocks=1 << 13, table_stride=1 << 13)), (BAD, dict(requests=None)), (MIS, dict(requests=FAKE + 2))])
def test_free_refusals(code, change):
    assert sar.topk_page_free(free_args(**change), 0) == code


@pytest.mark.parametrize("code, change", POOL + [
    (BAD, dict(max_copies=-1)), (BAD, dict(table_out_stride=7)), (BAD, dict(source=None)), (BAD, dict(target=None)), (BAD, dict(block_table_out=None)), (BAD, dict(shares_out=None)),
    (BAD, dict(free_blocks_out=None)), (BAD, dict(taken_out=None)), (BAD, dict(scratch=None)), (SMALL, dict(scratch_bytes=135)), (MIS, dict(scratch=FAKE + 4)), (MIS, dict(taken_out=FAKE + 2))])
def test_compact_refusals(code, change):
    assert sar.topk_page_compact(compact_args(**change), 0) == code


@pytest.mark.parametrize("code, change", [
    (BAD, dict(num_copies=-1)), (BAD, dict(num_caches=-1)), (BAD, dict(num_caches=257)), (BAD, dict(caches=None)), (BAD, dict(source=None)), (BAD, dict(target=None)), (BAD, dict(workspace=None)),
    (BAD, dict(num_blocks=-1)), (BAD, dict(n0=0)), (BAD, dict(n1=0)), (BAD, dict(run_bytes=0)), (BAD, dict(base=None)), (UNS, dict(run_bytes=1 << 36)), (UNS, dict(n0=1 << 20, n1=1 << 12)),
    (MIS, dict(source=FAKE + 2)), (MIS, dict(target=FAKE + 1)), (MIS, dict(workspace=FAKE + 8))])
def test_copy_refusals(code, change):
    assert sar.topk_page_copy(copy_args(**change), 0) == code


def test_nothing_to_do_is_no_work():
    assert sar.topk_block_means(means_args(num_requests=0, k=None), 0) == sar.TOPK_OK
    assert sar.topk_block_scores(scores_args(num_rows=0, q=None), 0) == sar.TOPK_OK
    assert sar.topk_block_attention(blocks_args(num_rows=0, q=None, blocks=None), 0) == sar.TOPK_OK
    assert sar.topk_shared_attention(shared_args(num_rows=0, q=None, scratch=None), 0) == sar.TOPK_OK
    assert sar.topk_page_fork(fork_args(num_forks=0, parents=None), 0) == sar.TOPK_OK
    assert sar.topk_page_free(free_args(num_freed=0, requests=None), 0) == sar.TOPK_OK
    assert sar.topk_page_copy(copy_args(num_copies=0, source=None), 0) == sar.TOPK_OK
    assert sar.topk_page_copy(copy_args(num_caches=0, source=None), 0) == sar.TOPK_OK


# ---- the Python side -------------------------------------------------------------------------------------------

@pytest.fixture
def dec():
    """A decoder whose device is that of CPU tensors, without a library call."""
    d = object.__new__(sar.PagedDecoder)
    d.device, d._dev = -1, "cpu"
    return d


def runs(dec, t):
    c = sar.TopkPageCache.from_buffer_copy(dec._page_cache(t))
    return [(b * c.block_stride + i * c.stride0 + j * c.stride1, c.run_bytes) for b in range(c.num_blocks) for i in range(c.n0) for j in range(c.n1)]


def test_caches_are_read_as_runs_of_bytes(dec):
    big = torch.zeros(5, 6, 4, 3, 8)
    for t, pieces in [(big, 1), (big.transpose(1, 3), 1), (big[:, :, :, 1], 24), (big[:, 2:4, 1:, :, ::2], None), (big[:, 1:3, :, :, :], 1), (big[:, :, 1:3], 6), (big[::2], 1),
                      (big[:, :, :, 1:, 3:], None), (torch.zeros(7), 1), (torch.zeros(4, 3).half(), 1), (big.permute(0, 4, 2, 1, 3), 1), (big[0], 1), (big.double()[:, :, ::3, :, 2:], None)]:
        if pieces is None and sum(n > 1 for n in t.shape[1:]) > 3:
            try:
                got = runs(dec, t)
            except ValueError:
                continue
        else:
            got = runs(dec, t)
        if pieces is not None:
            assert len(got) == pieces * len(t)
        size = t.element_size()
        places = sorted(x * size for x in torch.arange(t.untyped_storage().nbytes() // size).as_strided(t.shape, t.stride()).flatten().tolist())
        assert sorted(at + i for at, n in got for i in range(0, n, size)) == places


@pytest.mark.parametrize("make", [lambda: torch.zeros(4, 1).expand(4, 8), lambda: torch.zeros(1, 8).expand(4, 8)[:, ::2], lambda: torch.zeros(()), lambda: torch.zeros(3, 0),
                                  lambda: torch.zeros(64).as_strided((4, 3, 4), (16, 2, 1)), lambda: torch.zeros(2, 8, 8, 8, 8)[:, ::2, ::2, ::2, ::2]])
def test_caches_that_are_refused(dec, make):
    with pytest.raises(ValueError):
        dec._page_cache(make())


# ---- the sources -------------------------------------------------------------------------------------------------

NEW = ["attention_forms.cuh", "block_attention.cu", "tail_attention.cu", "prefix_attention.cu", "whole_attention.cu", "shared_attention.cu", "wide_prefix.cu", "attention_parts.cuh", "block_scores.cu"]


@pytest.mark.parametrize("name", NEW)
def test_kernels_use_the_wrappers(name):
    assert not source.ALIGNED.search(source.source(name))


def test_the_clusters_barrier_brings_the_warp_together_first():
    text = source.source("pages.cu")
    bodies = [b for b in source.functions(text).values() if source.ALIGNED.search(b)]
    assert len(bodies) == 2 and all(b.strip().startswith("__syncwarp();") for b in bodies) and len(source.ALIGNED.findall(text)) == 2


@pytest.mark.parametrize("name", NEW + ["pages.cu"])
def test_no_loads_for_data_that_nothing_writes(name):
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", source.source(name))


@pytest.mark.parametrize("name", [n for n in NEW if n.endswith(".cu")] + ["pages.cu"])
def test_every_kernel_waits_for_the_one_before(name):
    text = source.source(name)
    for body in re.findall(r"^__global__.*?^\}", text, re.M | re.S):
        assert "dependent_wait();\n  dependent_launch();" in body
