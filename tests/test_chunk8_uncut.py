"""How the chunk attention shares out sequences of a few key tiles, which are not cut,
from the header that the kernel is compiled with, on the host under the
undefined-behaviour sanitiser."""
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
  if (!std::strcmp(argv[1], "limit")) {  // max_seqlen: whether it is cut, and the most tiles of an item then
    const int keys = std::atoi(argv[2]);
    std::printf("%%d %%d\\n", uncut(keys), tiles(keys));
    return 0;
  }
  // CTAs of the launch, items as tiles:dual,...: each CTA's items, and the tiles of each that are its
  const int most = std::atoi(argv[1]);
  int nt[4096], w[4096], n = 0;
  long long counted_tiles = 0, all = 0;
  for (char* q = argv[2]; *q; ++n) {
    nt[n] = std::strtol(q, &q, 10);
    w[n] = std::strtol(q + 1, &q, 10);  // (for now: dual)
    counted_tiles += counted(nt[n], true);
    if (*q == ',') ++q;
  }
  for (int i = 0; i < n; ++i) all += (w[i] = tile_units(w[i] != 0, few(counted_tiles, most))) * counted(nt[i], true);
  const int ctas = runs(all, most), extra = extra_units(all, ctas);
  const long long total = all + static_cast<long long>(extra) * n;
  std::printf("%%d %%lld\\n", ctas, total);
  for (int c = 0; c < ctas; ++c) {
    const long long lo = run_start(c, total, ctas), hi = run_start(c + 1LL, total, ctas);
    long long first = 0;
    for (int i = 0; i < n; ++i) {
      first += extra;
      const int k0 = tiles_before(lo - first, w[i], nt[i], true), k1 = tiles_before(hi - first, w[i], nt[i], true);
      if (k1 > k0) std::printf("%%d %%d %%d %%d %%d\\n", c, i, k0, k1, run_of(first, total, ctas));
      first += w[i];
    }
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("uncut")
    (d / "uncut.cpp").write_text(CODE % HEADER)
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-o", str(d / "uncut"),
                    str(d / "uncut.cpp")], check=True)

    def run(*args):
        out = subprocess.run([str(d / "uncut"), *map(str, args)], check=True, capture_output=True, text=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]

    return run


@pytest.mark.parametrize("most", [1, 2, 7, 152])
@pytest.mark.parametrize("items", [[(1, 1)], [(3, 0)], [(3, 1)], [(1, 1), (2, 0), (3, 1)], [(1 + i % 3, i % 2) for i in range(152)],
                                   [(1 + i % 3, i % 2) for i in range(153)], [(3, 0)] * 151 + [(1, 1)], [(1, 1)] * 1000,
                                   [(3, 0)] * 1000, [(1 + i % 3, int(i % 5 > 1)) for i in range(2000)]])
def test_an_item_is_whole_in_one_run(program, items, most):
    """Nothing is left to join: an item's tiles are all of them in the run in which it
    begins.  Items that can have a CTA each have one; more are spread evenly."""
    out = program(most, ",".join(f"{n}:{d}" for n, d in items))
    (ctas, total), rows = out[0], out[1:]
    assert 1 <= ctas <= most
    assert sorted(i for _, i, _, _, _ in rows) == list(range(len(items)))
    assert all((k0, k1) == (0, items[i][0]) and c == begins for c, i, k0, k1, begins in rows)
    assert [i for _, i, _, _, _ in sorted(rows)] == list(range(len(items)))  # in order
    load = [sum(c == x for x, *_ in rows) for c in range(ctas)]
    if len(items) <= most:
        assert load == [1] * len(items)
    else:
        # two units an item of one half and three of others, and the fixed cost: first units are
        # at least 2 + cost apart, so a run of L units has at most (L - 1) / (2 + cost) + 1 of them
        all_units = sum(2 if d else 3 for _, d in items)
        assert ctas == min(most, all_units // 3)
        cost = (total - all_units) // len(items)
        assert max(load) <= (-(-total // ctas) - 1) // (2 + cost) + 1


def test_limit(program):
    """A copying warp's page indexes (32 a step, eight of a tile at the most) reach over
    the tiles of an item that is not cut."""
    for keys, want in ((1, [1, 1]), (128, [1, 1]), (129, [1, 2]), (384, [1, 3]), (385, [0, 4]), (2 ** 31 - 1, [0, 2 ** 24])):
        assert program("limit", keys) == [want]
    assert 3 * 8 <= 32
