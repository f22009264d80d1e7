"""The attention kernels' arithmetic on numbers of tiles, compiled for the host (no GPU needed)."""
import os
import subprocess

import pytest

from sparse_attention_row_gb300 import build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_row_gb300", "csrc")


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    """A program that answers "x per" with group_of(x, per)."""
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cu").write_text('#include <cstdio>\n#include "attention_parts.cuh"\nint main() {\n  long long x, per;\n'
                                '  while (std::scanf("%lld %lld", &x, &per) == 2) std::printf("%lld\\n", static_cast<long long>(ltk::paged::group_of(x, per)));\n}\n')
    subprocess.check_call([build._nvcc(), "-std=c++17", "-O1", "-I", CSRC, "-o", str(d / "parts"), str(d / "parts.cu")])
    return lambda pairs: [int(x) for x in subprocess.run([str(d / "parts")], input="\n".join(f"{x} {per}" for x, per in pairs), capture_output=True, text=True, check=True).stdout.split()]


def test_groups_of_tiles_of_any_size(parts):
    # a group's tiles times key-value heads: 2^23 times 1024 at most, where 32 bits would be zero, or a few
    sizes = [1, 2, 7, 1000, 2 ** 22 - 1, 2 ** 22, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 23 * 513, 2 ** 33]
    places = [0, 1, 6, 7, 999, 2 ** 22 - 1, 2 ** 22, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 40 + 5]
    pairs = [(x, per) for per in sizes for x in places]
    assert parts(pairs) == [x // per for x, per in pairs]
