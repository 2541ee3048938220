// Which tiles the segments of the ragged products have, in whole numbers: on
// the device for the kernels, and on the host for whoever checks them.
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

}  // namespace bsq
