"""The chunk attention's arithmetic at its limits, from the header that the kernel is
compiled with, on the host under the undefined-behaviour sanitiser."""
import os
import random
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
