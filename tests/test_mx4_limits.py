"""Tiles of 16 rows and the 32 bits that a wave counts tiles in (csrc/moe_index.h, csrc/mx4_index.h), on the host.  CPU
only."""
import shutil
import subprocess

import pytest

from test_moe_index import CSRC, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")


def test_tiles_of_16_rows_up_to_the_most_rows_that_take_them(tmp_path):
    """64 lanes' counts stay below 2^32 for the most rows that tiles of each height may be cut from, whatever the
    offsets, and would not for twice as many; tiles and segments are as for the higher ones."""
    _run(tmp_path, r"""
        std::mt19937 g(3);
        EXPECT(rows_counted(32) == kMaxRows && rows_counted(16) < kMaxRows, "rows");
        auto check = [&](auto tm) {
          constexpr int TM = decltype(tm)::value;
          const int64_t most = rows_counted(TM) < kMaxRows ? rows_counted(TM) : kMaxRows;
          for (int64_t cap : {int64_t(40), int64_t(65536), most - 1, most})
            for (int E : {1, 2, 63, 64, 65, 1024}) {
              EXPECT(uint64_t(64) * uint64_t(cap / TM + E + 1) < uint64_t(1) << 32, "%lld rows", (long long)cap);
              for (int kind = 0; kind < 4; ++kind) {
                std::vector<int32_t> o(E + 1);
                for (int i = 0; i <= E; ++i)
                  o[i] = kind == 0 ? (i & 1 ? int32_t(cap) : 0) : kind == 1 ? (i & 1 ? INT32_MAX : INT32_MIN)
                       : kind == 2 ? int32_t(g()) : (i ? int32_t(cap) : 0);
                Wave<TM> w(Segments<TM>{o.data(), E, cap});
                EXPECT(w.total >= 0 && w.total <= cap / TM + E + 1, "%d tiles of %d rows", w.total, TM);
                for (int rep = 0; rep < 100 && w.total > 0; ++rep) {
                  const int mt = rep == 0 ? 0 : rep == 1 ? w.total - 1 : int(g() % unsigned(w.total));
                  const Segment s = w.at(mt);
                  EXPECT(s.e >= 0 && s.e <= E && s.row0 >= 0 && s.row0 < s.end && s.end <= cap, "tile %d", mt);
                }
              }
            }
          EXPECT(uint64_t(64) * uint64_t(2 * rows_counted(TM) / TM + 2) >= uint64_t(1) << 32, "a bound that is far off");
        };
        check(std::integral_constant<int, 16>{});
        check(std::integral_constant<int, 32>{});
    """)


MAIN = r"""
#include <cmath>
#include <cstdio>
#include <random>
#include "mx4_index.h"
using namespace bsq;
#define EXPECT(c, ...) do { if (!(c)) { printf("%s: ", #c); printf(__VA_ARGS__); printf("\n"); return 1; } } while (0)
int main() {
  std::mt19937_64 g(4);
  auto between = [&](double lo, double hi) { return int64_t(lo * pow(hi / lo, double(g() >> 11) / double(1ull << 53))); };
  int few = 0;
  for (int i = 0; i < 300000; ++i) {
    const int64_t cap = i % 7 ? between(1, double(kMaxRows)) : kMaxRows - int64_t(g() % 1000);
    const int64_t E = 1 + int64_t(g() % 1024), N = 16 * between(1, i % 3 ? 16 : 1 << 26), k = between(1, 0x7FFFFFFF);
    const int64_t T = i % 2 ? between(1, 1 << 30) : cap, K = 32 * between(1, 1 << 19);
    if (cap / 16 + E + 1 > 0x7FFFFFFF / ((N + 15) / 16 + 1)) continue;  // refused
    const Mx4Size s{true, i % 4 < 2, T, cap, E, k, N, K};
    const Mx4Tile t = mx4_tile(s);
    const bool is_few = t == Mx4Tile::few16x16 || t == Mx4Tile::few16x32 || t == Mx4Tile::few32x32;
    few += is_few;
    EXPECT(!is_few || cap <= rows_counted(16), "cap %lld E %lld N %lld", (long long)cap, (long long)E, (long long)N);
    // tiles of E segments and a tail of cap rows in all
    for (int64_t tm : {16, 32, 64, 128, 256}) {
      int64_t rows = cap, tiles = 0;
      for (int64_t e = 0; e <= E && rows > 0; ++e) {
        const int64_t n = e == E ? rows : g() % 2 ? 1 + int64_t(g() % uint64_t(rows)) : 1;
        tiles += (n + tm - 1) / tm;
        rows -= n;
      }
      EXPECT(s.launched(tm, 16) >= tiles * ((N + 15) / 16), "%lld tiles", (long long)tiles);
      EXPECT(s.launched(tm, 16) <= (cap / tm + E + 1) * ((N + 15) / 16), "more than the limit");
    }
  }
  EXPECT(few > 1000, "%d sizes", few);
  puts("ok");
}
"""


def test_few_rows_kernels_are_taken_within_that(tmp_path):
    """No size that the call accepts takes a kernel of 16-row tiles past the rows that those are counted for, and a launch
    has a workgroup for each tile of any split."""
    (tmp_path / "few.cpp").write_text(MAIN)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow",
                        "-fno-sanitize-recover=all", "-I", CSRC, str(tmp_path / "few.cpp"), "-o", str(tmp_path / "few")],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(tmp_path / "few")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
