"""The chunk attention's arithmetic on rows, tiles and runs, from the header that the
kernel is compiled with, on the host under the undefined-behaviour sanitiser."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "io_aware_attention_flash_gb300", "csrc", "chunk8_items.h")

CODE = """
#include <cstdio>
#include <cstdlib>
#include "%s"
using namespace fa::chunk8;
int main(int argc, char** argv) {
  if (argc == 6) {  // len n G causal row-blocks: each block's tiles, whole and by halves, and the rows' keys
    const int len = std::atoi(argv[1]), n = std::atoi(argv[2]), G = std::atoi(argv[3]), causal = std::atoi(argv[4]);
    for (int rb = 0; rb < std::atoi(argv[5]); ++rb)
      std::printf("%%d %%d %%d\\n", row_tiles(len, n, G, rb * kRows, kRows, causal), row_tiles(len, n, G, rb * kRows, kHalf, causal),
                  row_tiles(len, n, G, rb * kRows + kHalf, kHalf, causal));
    std::printf("%%d %%d\\n", visible(len, n, 0, causal), visible(len, n, n - 1, causal));
  } else if (argc == 4) {  // tiles ctas 0: the units before an item's first tile
    std::printf("%%d\\n", extra_units(std::atoll(argv[1]), std::atoll(argv[2])));
  } else {  // total ctas: the runs' beginnings, and the run of each run's first and last unit
    const long long total = std::atoll(argv[1]), ctas = std::atoll(argv[2]);
    for (long long c = 0; c < ctas; ++c)
      std::printf("%%lld %%d %%d\\n", run_start(c, total, ctas), run_of(run_start(c, total, ctas), total, ctas),
                  run_of(run_start(c + 1, total, ctas) - 1, total, ctas));
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("items")
    (d / "items.cpp").write_text(CODE % HEADER)
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-o", str(d / "items"),
                    str(d / "items.cpp")], check=True)

    def run(*args):
        out = subprocess.run([str(d / "items"), *map(str, args)], check=True, capture_output=True, text=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]

    return run


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("G", [1, 3, 7, 40, 300])
@pytest.mark.parametrize("length,n", [(0, 3), (1, 1), (5, 9), (128, 128), (129, 128), (1000, 300), (2 ** 31 - 1, 1), (2 ** 31 - 1, 700)])
def test_tiles_cover_what_the_rows_see(program, length, n, G, causal):
    blocks = -(-n * G // 256) + 1
    out = program(length, n, G, causal, blocks)
    see = lambda i: max(0, min(length, length - n + i + 1)) if causal else length  # noqa: E731

    def tiles(first, count):
        rows = range(first, min(first + count, n * G))
        return max(max(1, -(-see(f // G) // 128)) for f in (rows[0], rows[-1])) if rows else 0

    for rb in range(blocks):
        assert out[rb] == [tiles(rb * 256, 256), tiles(rb * 256, 128), tiles(rb * 256 + 128, 128)]
    assert out[-1] == [see(0), see(n - 1)]


@pytest.mark.parametrize("total", [1, 2, 151, 152, 153, 1000, 123457, 2 ** 40 + 12345, 2 ** 55 - 1])
def test_runs_are_even_and_found_again(program, total):
    ctas = min(152, total)
    out = program(total, ctas)
    starts = [row[0] for row in out] + [total]
    assert starts[0] == 0 and all(total // ctas <= b - a <= -(-total // ctas) for a, b in zip(starts, starts[1:]))
    assert [row[1:] for row in out] == [[c, c] for c in range(ctas)]


@pytest.mark.parametrize("tiles,ctas", [(1, 1), (7, 7), (152, 152), (303, 152), (304, 152), (455, 152), (456, 152), (10 ** 9, 152)])
def test_units_before_an_item(program, tiles, ctas):
    """No more than a CTA has tiles, so that no run is all fixed cost where work is scarce."""
    (extra,), = program(tiles, ctas, 0)
    assert 0 <= extra <= 3 and extra < tiles / ctas and (extra == 3 or extra == tiles // ctas - 1)
