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
  } else if (argc == 4) {  // most, "cut", items as nt:w,...: every CTA's tiles of every item it has any of
    const int most = std::atoi(argv[1]);
    int nt[4096], w[4096], n = 0;
    long long all = 0;
    for (char* q = argv[3]; *q; ++n) {
      nt[n] = std::strtol(q, &q, 10);
      w[n] = std::strtol(q + 1, &q, 10);
      all += static_cast<long long>(nt[n]) * w[n];
      if (*q == ',') ++q;
    }
    long long tiles = 0;
    for (int i = 0; i < n; ++i) tiles += nt[i];
    if (few(tiles, most)) {  // all tiles count the same
      all = 0;
      for (int i = 0; i < n; ++i) all += static_cast<long long>(nt[i]) * (w[i] = tile_units(w[i] == 2, true));
    }
    const int ctas = runs(all, most), extra = extra_units(all, ctas);
    const long long total = all + static_cast<long long>(extra) * n;
    std::printf("%%d %%d %%lld\\n", ctas, extra, total);
    for (int c = 0; c < ctas; ++c) {
      const long long lo = run_start(c, total, ctas), hi = run_start(c + 1, total, ctas);
      long long first = 0;
      for (int i = 0; i < n; ++i) {
        first += extra;
        const int k0 = tiles_before(lo - first, w[i], nt[i], false), k1 = tiles_before(hi - first, w[i], nt[i], false);
        if (k1 > k0) std::printf("%%d %%d %%d %%d %%d %%d\\n", c, i, k0, k1, run_of(first, total, ctas),
                                 run_of(first + static_cast<long long>(nt[i] - 1) * w[i], total, ctas));
        first += static_cast<long long>(nt[i]) * w[i];
      }
    }
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


@pytest.mark.parametrize("most", [1, 3, 152])
@pytest.mark.parametrize("items", [[(1, 2)], [(1, 3)], [(7, 2)], [(7, 3)], [(3, 3), (1, 2), (2, 3), (5, 2)], [(1, 2)] * 300,
                                   [(256, 2)] * 32, [(1 + i % 9, 2 + i % 2) for i in range(500)], [(250, 3)] * 256, [(2, 3), (1, 2)] * 40, [(1, 2)] * 152, [(1, 2)] * 153])
def test_every_tile_is_in_one_run(program, items, most):
    """And the CTAs between an item's first and last all have tiles of it, which the join relies on."""
    out = program(most, "cut", ",".join(f"{n}:{w}" for n, w in items))
    (ctas, extra, total), rows = out[0], out[1:]
    assert 1 <= ctas <= most and 0 <= extra <= 18
    if sum(n for n, _ in items) <= most:  # a CTA for each tile
        assert ctas == sum(n for n, _ in items) and all(k1 - k0 == 1 for _, _, k0, k1, _, _ in rows)
    seen = {}
    for c, i, k0, k1, c0, c1 in rows:
        assert k0 == seen.get(i, (0, 0))[0]
        parts = seen.get(i, (0, []))[1] if i in seen else []
        seen[i] = (k1, parts + [c])
        assert c0 <= c <= c1
        seen[i] = (k1, parts + [c])
        assert (k0 == 0) == (c == c0) and (k1 == items[i][0]) == (c == c1)
    assert len(seen) == len(items)
    for i, (end, parts) in seen.items():
        assert end == items[i][0] and parts == list(range(parts[0], parts[-1] + 1))
    if most == 152 and len(items) > 200:  # and the runs are even, whole tiles and an item's cost apart
        cost = {}
        for c, i, k0, k1, _, _ in rows:
            cost[c] = cost.get(c, 0) + (k1 - k0) * items[i][1] + (extra if k0 == 0 else 0)
        assert max(cost.values()) <= total / ctas + extra + 3
