"""The cache attention's arithmetic on lengths, from the header that the kernel is
compiled with, on the host under the undefined-behaviour sanitiser: for lengths up
to 2^31 - 1, no lane takes a page behind the last token's for one of the sequence."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "io_aware_attention_flash_gb300", "csrc", "cache8_tiles.h")

# Walks the last tiles of a length as the kernel does: a unit of 32 pages, one a
# lane, and each row's tokens in the tile.
CODE = """
#include <cstdio>
#include <cstdlib>
#include "%s"
using namespace fa::cache8;
int main(int argc, char** argv) {
  const int len = std::atoi(argv[1]), tokens = std::atoi(argv[2]), shift = std::atoi(argv[3]);
  const int nt = tiles_of(len, tokens), pages = pages_of(len, shift), ppt = tokens >> shift;
  std::printf("%%d %%d\\n", nt, pages);
  for (int kt = nt > 40 ? nt - 40 : 0; kt < nt; ++kt) {
    for (int lane = 0; lane < 32; ++lane) std::printf("%%d ", kt * ppt + lane < pages ? 1 : 0);
    for (int row = 0; row < tokens; ++row) std::printf("%%d ", tokens_from(len, kt, tokens, row));
    std::printf("\\n");
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("tiles")
    (d / "walk.cpp").write_text(CODE % HEADER)
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-o", str(d / "walk"),
                    str(d / "walk.cpp")], check=True)
    return str(d / "walk")


@pytest.mark.parametrize("shift", [4, 5, 6, 7])
@pytest.mark.parametrize("tokens", [128, 256])
@pytest.mark.parametrize("length", [0, 1, 255, 256, 257, 100000, 2 ** 31 - 300, 2 ** 31 - 257, 2 ** 31 - 256, 2 ** 31 - 129,
                                    2 ** 31 - 128, 2 ** 31 - 2, 2 ** 31 - 1])
def test_ends(program, length, tokens, shift):
    out = subprocess.run([program, str(length), str(tokens), str(shift)], check=True, capture_output=True, text=True)
    rows = [[int(x) for x in line.split()] for line in out.stdout.splitlines()]
    nt, pages = -(-length // tokens), -(-length // 2 ** shift)
    assert rows[0] == [nt, pages]
    ppt = tokens >> shift
    for kt, row in zip(range(max(0, nt - 40), nt), rows[1:]):
        assert row[:32] == [int(kt * ppt + lane < pages) for lane in range(32)]
        assert row[32:] == [length - kt * tokens - r for r in range(tokens)]


def test_the_kernel_has_no_other_arithmetic_on_lengths():
    """What a length is added to or compared with goes through the functions above."""
    code = open(os.path.join(os.path.dirname(HEADER), "fa_cache8.cu")).read()
    for bad in ("+ p.block - 1", "* p.block <", "kTokens<D> - 1", "+ NP * r)"):
        assert bad not in code, bad
