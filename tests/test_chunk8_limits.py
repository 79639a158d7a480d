"""The chunk attention's arithmetic at its limits, from the header that the kernel is
compiled with, on the host under the undefined-behaviour sanitiser."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "io_aware_attention_flash_gb300", "csrc", "chunk8_items.h")

CODE = """
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "%s"
using namespace fa::chunk8;
int main(int argc, char** argv) {
  if (!std::strcmp(argv[1], "reach")) {  // len all n causal row...: keys that the rows see
    const int len = std::atoi(argv[2]), all = std::atoi(argv[3]), n = std::atoi(argv[4]), causal = std::atoi(argv[5]);
    for (int i = 6; i < argc; ++i) std::printf("%%d\\n", visible(reach(len, all, n, causal), n, std::atoi(argv[i]), causal));
  } else if (!std::strcmp(argv[1], "last")) {  // n G row-block...: whether it is the last
    for (int i = 4; i < argc; ++i) std::printf("%%d\\n", last_block(std::atoi(argv[2]), std::atoi(argv[3]), std::atoi(argv[i])));
  } else if (!std::strcmp(argv[1], "walk")) {  // G, the sequences' new tokens: the pairs from the first with rows on
    const int G = std::atoi(argv[2]), B = argc - 3;
    auto next_with = [&](int b) {
      while (b < B && std::atoi(argv[3 + b]) == 0) ++b;
      return b;
    };
    int b = next_with(0), rb = 0;
    while (b < B) {
      std::printf("%%d %%d\\n", b, rb);
      next_pair(b, rb, std::atoi(argv[3 + b]), G, next_with);
    }
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("limits")
    (d / "limits.cpp").write_text(CODE % HEADER)
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-o", str(d / "limits"),
                    str(d / "limits.cpp")], check=True)

    def run(*args):
        out = subprocess.run([str(d / "limits"), *map(str, args)], check=True, capture_output=True, text=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]

    return run


MOST = 2 ** 31 - 1


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("length,new,max_new", [
    (100, 10, 7), (100, 100, 1), (5, 10, 7), (1, 10, 7), (0, 10, 9), (100, 7, 7), (100, 3, 7), (MOST, MOST, 1), (MOST, MOST, MOST - 1),
    (0, MOST, 1), (3, MOST, MOST - 1), (MOST, 1, 1)])
def test_rows_below_max_new_see_what_they_see_of_the_whole(program, length, new, max_new, causal):
    n = min(new, max_new)
    rows = sorted({0, n // 2, n - 1})
    want = [max(0, min(length, length - new + i + 1)) if causal else length for i in rows]
    assert [x[0] for x in program("reach", length, new, n, causal, *rows)] == want


@pytest.mark.parametrize("G", [1, 3, 8, 256, 300])
@pytest.mark.parametrize("new", [[1], [0, 0, 5, 0], [4096] + [1] * 50 + [0] * 200 + [256, 257, 0, 255], [0] * 3000 + [100000, 0, 0, 33],
                                 [300, 0, 512, 85, 86]])
def test_pairs_with_rows_are_gone_through_without_the_others(program, new, G):
    """As many steps as there are such pairs: a copying warp that stepped over the empty
    ones, the longest sequence's row blocks for each other sequence, could keep the CTA's
    waits past their limit (2^25 pairs of two loads each and a division: seconds)."""
    new = [min(n, (2 ** 31 - 1) // G) for n in new]
    assert program("walk", G, *new) == [[b, rb] for b, n in enumerate(new) for rb in range(-(-n * G // 256))]


@pytest.mark.parametrize("n,G", [(MOST, 1), (1, MOST), (MOST // 300, 300), (2 ** 23, 255)])
def test_last_row_block_at_the_ends_of_int(program, n, G):
    last = (n * G - 1) // 256
    assert program("last", n, G, last - 1, last) == [[0], [1]]
