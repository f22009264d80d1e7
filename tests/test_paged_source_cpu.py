"""What the paged kernels' sources have to keep to, where a run cannot show it: the compiler may make good for a breach
today and not tomorrow."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_row_gb300", "csrc")
PAGED = ["kv_map.cu", "index_logits.cu", "paged_attention.cu", "cache_map.cu", "cache_map.cuh", "token_copies.cuh", "paged.cuh", "umma.cuh"]
ALIGNED = re.compile(r"\.aligned|\bbar\.sync")


def source(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def functions(text):
    """The bodies of the functions that begin in the first column, by their first line."""
    found = {}
    for m in re.finditer(r"^(?:static )?__device__[^\n;]*\{ *\n(.*?)^\}", text, re.M | re.S):
        found[m.group(0).split("\n")[0]] = m.group(1)
    return found


def test_instructions_of_a_whole_warp_bring_it_together_first():
    # PTX: the behaviour of an .aligned instruction is undefined unless all threads of the warp execute it together
    whole = source("umma.cuh")
    seen = 0
    for head, body in functions(whole).items():
        if not ALIGNED.search(body):
            continue
        before = body[:ALIGNED.search(body).start()]
        assert "__syncwarp();" in before, head
        rest = body[body.index("__syncwarp();"):]
        assert not re.search(r"\b(while|mbar_\w+)\b|\bif \(|\?", rest), f"{head}: something may split the warp again"
        seen += len(ALIGNED.findall(body))
    assert seen == len(ALIGNED.findall(whole)) > 0


@pytest.mark.parametrize("name", [n for n in PAGED if n != "umma.cuh"])
def test_kernels_use_the_wrappers(name):
    assert not ALIGNED.search(source(name))


@pytest.mark.parametrize("name", PAGED + ["topk_short.cu", "topk_sort.cu"])
def test_no_loads_for_data_that_nothing_writes(name):
    # ld.global.nc, which __ldg() is, wants memory that is constant while the kernel runs. These kernels begin before the one
    # that writes their block table, lengths, scales or logits has ended.
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", source(name))
