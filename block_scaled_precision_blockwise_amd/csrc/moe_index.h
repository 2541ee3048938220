// Whole numbers of the expert-layer calls, on the device for the kernels and on
// the host for the launches and for whoever checks them: the parts that large
// calls are launched in, which tiles the segments of the ragged products have,
// and which size of tile a product takes.
// Nothing here trusts the offsets: whatever they hold, no number passes 32
// bits and no row lies outside the arrays.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define BSQ_INDEX __host__ __device__ __forceinline__
#else
#define BSQ_INDEX inline
#endif

namespace bsq {

BSQ_INDEX int bounded(int v, int64_t cap) { return v < 0 ? 0 : (v > cap ? int(cap) : v); }

// A launch has less than 2^32 threads.  Calls of one workgroup to a few tokens
// are cut into launches of at most kLaunchTokens tokens (a multiple of 16, so
// that every part of an array that is aligned is), calls of one to a tile or a
// run of elements into launches of at most kLaunchGroups.
constexpr int64_t kMaxThreads = 0xFFFFFFFF;
constexpr int64_t kLaunchTokens = int64_t(1) << 24;
constexpr int64_t kLaunchGroups = int64_t(1) << 22;  // of 256 or 512 threads
// f(first, count) for each part; ends with the first status that is not zero.
template <typename F>
auto in_parts(int64_t n, int64_t most, F&& f) -> decltype(f(n, n)) {
  decltype(f(n, n)) s{};
  for (int64_t at = 0; at < n && int(s) == 0; at += most) s = f(at, n - at < most ? n - at : most);
  return s;
}

// Rows that the products' arrays may have: 64 lanes with `limit` tiles each
// stay below 2^32.
constexpr int64_t kMaxRows = 0x7FFFFFFF - 0xFFFF;

// Whether row r of a tile whose first row is row0 is before `end`.
BSQ_INDEX bool row_in(int row0, int r, int end) { return r < end - row0; }

// Byte of column n0 of row row0 + r of an array with `pitch` bytes to a row and
// `elem` to a column.
BSQ_INDEX int64_t byte_at(int row0, int r, int64_t pitch, int n0, int elem) {
  return (int64_t(row0) + r) * pitch + int64_t(n0) * elem;
}

// A tile's segment (E: the rows past the last), first row and segment's end.
struct Segment {
  int e, row0, end;
};

// The segments [offsets[i], offsets[i + 1]) of i = 0 .. E - 1, and as segment E
// the rows past the last, each cut into tiles of TM (32 or more) rows from its
// first row.  A wave's lane l has c segments from l c on.
template <int TM>
struct Segments {
  const int32_t* offsets;
  int E;
  int64_t cap;

  BSQ_INDEX int lo(int i) const { return bounded(offsets[i], cap); }
  BSQ_INDEX int hi(int i) const { return i < E ? bounded(offsets[i + 1], cap) : int(cap); }
  BSQ_INDEX int share() const { return (E + 64) / 64; }
  BSQ_INDEX int end(int lane) const { return (lane + 1) * share() < E + 1 ? (lane + 1) * share() : E + 1; }
  static BSQ_INDEX int tiles(int lo, int hi) { return hi > lo ? (hi - lo - 1) / TM + 1 : 0; }
  // No more than these where the offsets ascend.  Others may ask for up to E
  // times as many, past 2^31: what passes the limit is not there.
  BSQ_INDEX int limit() const { return int(cap / TM) + E + 1; }
  // Tiles of a lane's segments, cut to the limit.
  BSQ_INDEX uint32_t lane_tiles(int lane) const {
    uint32_t n = 0;
    for (int i = lane * share(); i < end(lane); ++i) {
      n += uint32_t(tiles(lo(i), hi(i)));
      if (n > uint32_t(limit())) n = uint32_t(limit());
    }
    return n;
  }
  // Whether tile mt is one of a lane's, which has `mine` after `before` of others.
  static BSQ_INDEX bool has(uint32_t before, uint32_t mine, int mt) { return uint32_t(mt) - before < mine; }
  // The `left`-th tile of a lane's segments.
  BSQ_INDEX Segment at(int lane, int left) const {
    for (int i = lane * share(); i < end(lane); ++i) {
      const int l = lo(i), h = hi(i), n = tiles(l, h);
      if (left < n) return Segment{i, l + left * TM, h};
      left -= n;
    }
    return Segment{E, int(cap), int(cap)};
  }
};

// ------------------------------------------------- which tiles a call takes --
constexpr int64_t kCUs = 256;

BSQ_INDEX int64_t up_to(int64_t v, int64_t m) { return (v + m - 1) / m; }

// Weight gradients: whether the experts' `per` tiles of 256 x 256 go to the
// XCDs in chunks of 32: chunks that are mostly full, experts that fit the lanes.
BSQ_INDEX bool dealt(int per, int E) {
  const int chunks = (per + 31) / 32;
  return E <= 64 && 8 * per >= 7 * 32 * chunks;
}

enum class MoeTile { t32x64, t64x64, t64x128s3, t64x128, t128x128s3, t128x128, t256x256, t256x256_stream };

inline MoeTile product_tile(int64_t T, int64_t cap, int64_t E, int64_t N, int64_t K, int64_t k, bool gathers) {
  // rows that hold a choice, as far as the host knows, and per expert
  const int64_t n = gathers && T < cap / k ? T * k : cap, rows = n / E;
  // us at (rows per expert, experts, N, K), 256 x 256 tiles against the next:
  // (256, 16, 2048, 2048) 32 / 41, (192, 64, 2048, 1024) 65 / 78; with fewer
  // tiles than most CUs (255, 8, 1792, 1024) 18.5 / 12.1.  The big tiles
  // address rows with 32 bits.
  if (rows >= 160 && (n / 256 + E / 2) * up_to(N, 256) >= 160 && T * K < (int64_t(1) << 32)) return MoeTile::t256x256;
  // Few tiles leave CUs idle: the smallest tiles of which no CU gets two (half
  // a part-full tile to an expert on average; rows that a plan's alignment
  // leaves empty count, as their workgroups start too).  us so / with 64 x 128
  // and two stages at (rows per expert, experts, N, K): 32 x 64 tiles (250, 4,
  // 256, 4096) 13 / 26, 64 x 64 (256, 4, 512, 4096) 16 / 26, 64 x 128 (250, 4,
  // 1536, 2048) 13 / 16; with more tiles than that, (325, 4, 1536, 2048), 64 x
  // 64 takes 19, 64 x 128 with three stages 18, with two 17
  auto few = [&](int64_t tm, int64_t tn) { return (cap / tm + (E + 1) / 2) * up_to(N, tn) <= kCUs; };
  if (few(32, 64)) return MoeTile::t32x64;
  if (rows >= 32) {
    if (few(64, 64)) return MoeTile::t64x64;
    // 64 x 128 against 128 x 128: (255, 8, 1792, 1024) 12.1 / 14.8, (192, 64,
    // 2048, 1024) 79 / 78; against 64 x 64: (37, 32, 2048, 1024, segments
    // aligned to 128) 26 / 32
    return few(64, 128) ? MoeTile::t64x128s3 : MoeTile::t64x128;
  }
  // few rows, where the weights' bytes are most of the work: three stages
  // against two (1, 32, 4096, 2048) 33 / 42; 32 rows against 64 (8, 32, 2048,
  // 1024) 13.8 / 16.4, (25, 32, 4096, 2048) 74 / 70
  return rows > 16 ? MoeTile::t64x64 : MoeTile::t32x64;
}

inline MoeTile wgrad_tile(int64_t cap, int64_t E, int64_t N, int64_t K) {
  // us with 256 x 256 tiles against 128 x 128 at (big tiles, rows per expert):
  // (128, 512) 20 / 17, (64, 8192) 85 / 60
  const int64_t big = up_to(N, 256) * up_to(K, 256) * E;
  if (big >= 256 && cap * 256 < (int64_t(1) << 32)) {
    // Where an XCD's chunk of 32 tiles reads more than its 4 MB of L2, one
    // operand is better off leaving it first.  us so / kept, (N, K, experts,
    // rows per expert): (2048, 2048, 16, 2048) 152 / 163, (2048, 2048, 8, 4096)
    // 136 / 147, (4096, 2048, 8, 4096) 248 / 270, (2048, 4096, 8, 4096) 280 /
    // 280, (2048, 1024, 16, 2048) 80 / 88; where it fits, (2048, 2048, 16,
    // 1125) 100 / 93, and where tiles are dealt by eighths, (1280, 2048, 12,
    // 2048) 117 / 107.  The products lose by it: 627 / 537.
    const int64_t across = up_to(K, 256), cols = across < 32 ? across : 32, rows = up_to(32, cols);
    const bool more = (rows + cols) * 256 * (cap / E) > (int64_t(4) << 20);
    return dealt(int(big / E), int(E)) && more ? MoeTile::t256x256_stream : MoeTile::t256x256;
  }
  // Few tiles leave CUs idle: the smallest tiles of which no CU gets two.  us
  // with 64 x 64 / 64 x 128 / 128 x 128 at (N, K, experts, rows per expert):
  // (512, 512, 4, 8192) 25 / 33 / 44, (1024, 512, 4, 8192) 45 / 36 / 44, (1024,
  // 768, 4, 4096) 48 / 43 / 34, (640, 640, 8, 4096) 64 / 46 / 36
  auto tiles = [&](int64_t tn, int64_t tk) { return up_to(N, tn) * up_to(K, tk) * E; };
  if (tiles(64, 64) <= kCUs) return MoeTile::t64x64;
  if (tiles(64, 128) <= kCUs) return MoeTile::t64x128s3;
  // a workgroup to a CU: three stages for it; more: two, so that two fit.  us
  // with three / two at (tiles, rows per expert): (256, 2048) 27 / 33, (256,
  // 8192) 48 / 60, (512, 512) 21 / 17
  return tiles(128, 128) <= kCUs ? MoeTile::t128x128s3 : MoeTile::t128x128;
}

}  // namespace bsq
