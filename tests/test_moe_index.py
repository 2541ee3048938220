"""The whole-number arithmetic of the ragged products (csrc/moe_index.h),
compiled for the host and run over offsets that no plan writes and over
arrays near the largest that the calls accept.  CPU only."""
import os
import shutil
import subprocess
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_blockwise_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")


def _run(tmp_path, body):
    """Compiles `body` (statements that call EXPECT) and runs it; signed
    overflow ends it."""
    src = tmp_path / "index.cpp"
    src.write_text(textwrap.dedent(r"""
        #include <cstdio>
        #include <cstdlib>
        #include <random>
        #include <type_traits>
        #include <vector>
        #include "moe_index.h"
        using namespace bsq;
        #define EXPECT(c, ...) do { if (!(c)) { printf("line %d: %s: ", __LINE__, #c); printf(__VA_ARGS__); printf("\n"); \
          exit(1); } } while (0)
        // What the 64 lanes of a wave make of the segments.
        template <int TM> struct Wave {
          Segments<TM> s; uint32_t before[64], mine[64]; int total;
          explicit Wave(Segments<TM> s_) : s(s_), total(0) {
            uint64_t sum = 0;
            for (int l = 0; l < 64; ++l) {
              before[l] = uint32_t(sum);
              sum += mine[l] = s.lane_tiles(l);
            }
            EXPECT(sum < uint64_t(1) << 32, "the lanes' sum");
            total = sum < uint64_t(s.limit()) ? int(sum) : s.limit();
          }
          Segment at(int mt) const {
            int found = -1;
            for (int l = 0; l < 64; ++l)
              if (s.has(before[l], mine[l], mt)) {
                EXPECT(found < 0, "tile %d in two lanes", mt);
                found = l;
              }
            EXPECT(found >= 0, "no lane has tile %d of %d", mt, total);
            return s.at(found, mt - int(before[found]));
          }
        };
        int main() {
    """) + textwrap.dedent(body) + "\nputs(\"ok\"); return 0; }\n")
    exe = tmp_path / "index"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow",
                        "-fno-sanitize-recover=all", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_tiles_of_ascending_offsets(tmp_path):
    """Every row is in one tile, in the order of the rows."""
    _run(tmp_path, r"""
        std::mt19937 g(1);
        auto check = [&](auto tm) {
          constexpr int TM = decltype(tm)::value;
          for (int E : {1, 2, 63, 64, 65, 300, 1024})
            for (int rep = 0; rep < 20; ++rep) {
              std::vector<int32_t> o(E + 1);
              int at = g() % 3;
              for (int i = 0; i <= E; ++i) { o[i] = at; at += g() % 4 == 0 ? g() % 700 : g() % 2; }
              const int64_t cap = o[E] + (rep % 2 ? g() % 500 : 0);
              Wave<TM> w(Segments<TM>{o.data(), E, cap});
              int row = o[0], mt = 0;
              for (; mt < w.total; ++mt) {
                const Segment s = w.at(mt);
                EXPECT(s.row0 == row && s.end > row && s.end <= cap, "tile %d: row %d, not %d", mt, s.row0, row);
                EXPECT(s.end == (s.e < E ? o[s.e + 1] : cap), "end of tile %d", mt);
                row = s.row0 + TM < s.end ? s.row0 + TM : s.end;
              }
              EXPECT(row == cap, "rows up to %d of %d", row, int(cap));
              EXPECT(w.total <= w.s.limit(), "%d tiles", w.total);
            }
        };
        check(std::integral_constant<int, 32>{});
        check(std::integral_constant<int, 64>{});
        check(std::integral_constant<int, 256>{});
    """)


def test_tiles_of_offsets_that_do_not_ascend(tmp_path):
    """Segments that overlap ask for up to E cap / tm tiles, past 2^31: there
    are no more than ascending ones can have, and each is inside the arrays."""
    _run(tmp_path, r"""
        std::mt19937 g(2);
        auto check = [&](auto tm) {
          constexpr int TM = decltype(tm)::value;
          for (int64_t cap : {int64_t(40), int64_t(65536), int64_t(1) << 27, (int64_t(1) << 27) + 77, int64_t(0x70000000)})
            for (int E : {2, 64, 65, 1024})
              for (int kind = 0; kind < 3; ++kind) {
                std::vector<int32_t> o(E + 1);
                for (int i = 0; i <= E; ++i)
                  o[i] = kind == 0 ? (i & 1 ? int32_t(cap) : 0) : kind == 1 ? (i & 1 ? INT32_MAX : INT32_MIN)
                                                                        : int32_t(g());
                Wave<TM> w(Segments<TM>{o.data(), E, cap});
                EXPECT(w.total >= 0 && w.total <= cap / TM + E + 1, "%d tiles of %d rows", w.total, TM);
                for (int rep = 0; rep < 200 && w.total > 0; ++rep) {
                  const int mt = rep == 0 ? 0 : rep == 1 ? w.total - 1 : int(g() % unsigned(w.total));
                  const Segment s = w.at(mt);
                  EXPECT(s.e >= 0 && s.e <= E && s.row0 >= 0 && s.row0 < s.end && s.end <= cap,
                         "tile %d: segment %d, rows %d .. %d", mt, s.e, s.row0, s.end);
                }
              }
        };
        check(std::integral_constant<int, 32>{});
        check(std::integral_constant<int, 64>{});
        check(std::integral_constant<int, 256>{});
    """)


def test_tiles_of_the_longest_segments(tmp_path):
    """One segment as long as the arrays may be: its tiles are all there, and a
    row of its last tile is inside if it is before the segment's end."""
    _run(tmp_path, r"""
        auto check = [&](auto tm) {
          constexpr int TM = decltype(tm)::value;
          for (int64_t cap : {kMaxRows, kMaxRows - 1, kMaxRows - TM + 1, int64_t(1) << 30})
            for (int E : {1, 3, 1024})
              for (int first : {0, 1, TM - 1, 70000}) {
                std::vector<int32_t> o(E + 1, int32_t(cap));
                o[0] = first;
                Wave<TM> w(Segments<TM>{o.data(), E, cap});
                const int want = int((cap - first + TM - 1) / TM);
                EXPECT(w.total == want, "%d tiles, not %d", w.total, want);
                const Segment s = w.at(want - 1);
                EXPECT(s.row0 == first + int64_t(want - 1) * TM && s.end == cap, "last tile at %d", s.row0);
                for (int r = 0; r < TM; ++r)
                  EXPECT(row_in(s.row0, r, s.end) == (int64_t(s.row0) + r < cap), "row %d of the last tile", r);
              }
        };
        check(std::integral_constant<int, 32>{});
        check(std::integral_constant<int, 64>{});
        check(std::integral_constant<int, 256>{});
        EXPECT(row_in(0x7FFFFFFF - 0xFFFF - 3, 2, 0x7FFFFFFF - 0xFFFF) && !row_in(0x7FFFFFFF - 40, 255, 0x7FFFFFFF), "rows");
    """)


def test_bytes_of_the_widest_outputs(tmp_path):
    """Columns up to 2^30 of 4 bytes, rows of 2^32 bytes: no product of them
    is cut to 32 bits."""
    _run(tmp_path, r"""
        for (int elem : {2, 4})
          for (int n0 : {0, 128, 1 << 29, (1 << 29) + 256, (1 << 30) - 128})
            for (int row0 : {0, 256, (1 << 30) - 256}) {  // of at most 2^60 elements
              const int64_t pitch = (int64_t(1) << 30) * elem;
              const __int128 want = (__int128(row0) + 128) * pitch + __int128(n0) * elem;
              EXPECT(byte_at(row0, 128, pitch, n0, elem) == want, "row %d, column %d of %d bytes", row0, n0, elem);
            }
    """)


def test_launches_are_cut_below_the_threads_that_one_has(tmp_path):
    """The parts cover every token once, in order; each is a launch that fits,
    of 4 tokens to a workgroup of 256 threads, or of workgroups of 512."""
    _run(tmp_path, r"""
        for (int64_t n : {int64_t(0), int64_t(1), kLaunchTokens, kLaunchTokens + 1, int64_t(67108865), int64_t(0x7FFFFFFF)}) {
          int64_t next = 0;
          in_parts(n, kLaunchTokens, [&](int64_t at, int64_t count) {
            EXPECT(at == next && count > 0 && at % 16 == 0, "part at %lld", (long long)at);
            EXPECT((count + 3) / 4 * 256 <= kMaxThreads, "%lld tokens", (long long)count);
            next = at + count;
            return 0;
          });
          EXPECT(next == n, "%lld of %lld tokens", (long long)next, (long long)n);
        }
        EXPECT(kLaunchGroups * 512 <= kMaxThreads && kLaunchGroups % 8 == 0, "workgroups");
        int calls = 0;
        EXPECT(in_parts(100, 10, [&](int64_t, int64_t) { return ++calls == 3 ? 7 : 0; }) == 7 && calls == 3, "status");
    """)


def test_the_gpu_tests_reach_every_tile(tmp_path):
    """The sizes of tests/test_gpu_moe_tiles.py take the tiles that they are
    named for, and these are all that a product or a weight gradient can take."""
    import test_gpu_moe_tiles as G

    lines, seen = [], (set(), set())
    for name, (lengths, N) in G.PRODUCT_TILES.items():
        cap, seen_in = sum(lengths) + 5, seen[0]
        seen_in.add(name)
        for steps in range(1, 10):
            lines.append(f"EXPECT(product_tile({cap}, {cap}, {len(lengths)}, {N}, {128 * steps}, 2, true) == MoeTile::{name}, "
                         f"\"{name} {steps}\");")
    for name, (blocks, all_blocks, N, K) in G.WGRAD_TILES.items():
        assert sum(blocks) <= all_blocks
        tile, *kind = name.split()
        seen[1].add(tile)
        big = -(-N // 256) * -(-K // 256)
        lines.append(f"EXPECT(wgrad_tile({128 * all_blocks}, {len(blocks)}, {N}, {K}) == MoeTile::{tile}, \"{name}\");")
        if tile.startswith("t256"):
            want = "false" if not kind and tile == "t256x256" else "true"
            lines.append(f"EXPECT(dealt({big}, {len(blocks)}) == {want}, \"{name}\");")
            if kind != ["one"] and kind != ["dealt"]:
                assert big * len(blocks) > 256  # workgroups that go through more than one tile
    assert seen[0] == {"t32x64", "t64x64", "t64x128s3", "t64x128", "t256x256"}
    assert seen[1] == {"t64x64", "t64x128s3", "t128x128s3", "t128x128", "t256x256", "t256x256_stream"}
    wild = [p.values for p in G.WILD]
    for (E, cap, N, K), name in zip(wild, ("t32x64", "t64x64", "t64x128s3", "t64x128", "t64x64", "t256x256", "t32x64")):
        lines.append(f"EXPECT(product_tile({cap}, {cap}, {E}, {N}, {K}, 2, true) == MoeTile::{name}, \"wild {N}\");")
        lines.append(f"EXPECT(product_tile({cap}, {cap}, {E}, {N}, {K}, 1, false) == MoeTile::{name}, \"wild {N}\");")
    _run(tmp_path, "\n".join(lines))
