// Which kernel a product with 4-bit weights takes, on the host for the launch
// and for whoever checks it.
#pragma once

#include "moe_index.h"

namespace bsq {

enum class Mx4Tile { few16x16, few16x32, few32x32, t32x64, t32x64g2, t64x64g2, t64x128g2, t64x128, t128x128, t256x256 };

// T rows to each of E products (dense), or cap rows of out over E experts, of
// which `gathers` tells that there are at most T k choices.
struct Mx4Size {
  bool ragged, gathers;
  int64_t T, cap, E, k, N, K;
  int64_t rows() const { return !ragged ? T * E : gathers && T < cap / k ? T * k : cap; }  // that count
  int64_t each() const { return ragged ? rows() / E : T; }
  // Tiles of tm x tn with work: of a segment's rows the last tile is part full.
  int64_t tiles(int64_t tm, int64_t tn) const {
    if (!ragged) return up_to(T, tm) * E * up_to(N, tn);
    const int64_t n = rows(), some = n < E ? n : E, t = n / tm + some * 3 / 5;
    return (t > some ? t : some) * up_to(N, tn);
  }
  // Tiles that are launched: those that any split over the experts can need.
  int64_t launched(int64_t tm, int64_t tn) const {
    return (ragged ? cap / tm + E + 1 : up_to(T, tm) * E) * up_to(N, tn);
  }
};

// Tiles of 16 x 16 up to which the kernels for few rows are taken.  No more rows
// than rows_counted(16) have as few.
constexpr int64_t kFewLaunched = 16 * kCUs;
static_assert(16 * kFewLaunched <= rows_counted(16), "a wave counts tiles in 32 bits");

inline Mx4Tile mx4_tile(const Mx4Size& s) {
  // Few tiles: the smallest of which no CU gets two.  Straight from memory to
  // registers, us of kernels in a replayed graph, weights from memory, against 32
  // x 64 tiles of two groups at (rows, N, K): 16 x 16 (1, 4096, 4096) 4.7 / 8.4,
  // (128, 256, 4096) 4.9 / 6.9; 16 x 32 (1, 8192, 4096) 6.1 / 8.8, (64, 2048,
  // 4096) 6.3 / 8.8; 32 x 32 (64, 4096, 2048) 5.2 / 5.9, and with weights that the
  // caches hold (64, 4096, 4096) 7.2 / 7.0.  Not where many workgroups start for
  // nothing, which also bounds the rows that their tiles of 16 are counted from.
  if (s.launched(16, 16) <= kFewLaunched) {
    if (s.tiles(16, 16) <= kCUs) return Mx4Tile::few16x16;
    if (s.tiles(16, 32) <= kCUs) return Mx4Tile::few16x32;
    if (s.tiles(32, 32) <= kCUs && s.K <= 2048) return Mx4Tile::few32x32;
  }
  // two groups of waves share a tile's contraction, inputs held by the caches: 32
  // x 64 against one group
  // (128, 4096, 4096) 7.2 / 8.6, 64 x 64 (1024, 1024, 16384) 22 / 29, 64 x 128
  // (1021, 1792, 2880) 13.8 / 17.8
  if (s.tiles(32, 64) <= kCUs) return Mx4Tile::t32x64g2;
  if (s.each() <= 32) return Mx4Tile::t32x64;  // 4 rows to each of 32 experts 36 us, 64 x 128 36, two groups 41
  if (s.tiles(64, 64) <= kCUs) return Mx4Tile::t64x64g2;
  if (s.tiles(64, 128) <= kCUs) return Mx4Tile::t64x128g2;
  // 64 x 128 against 128 x 128 at (rows to each, experts, N, K): (64, 32, 2048,
  // 1024) 15 / 21, (128, 32, 2048, 2048) 31 / 30, (2048, 1, 2048, 2048) 10.9 / 10.5
  const int64_t mid = s.tiles(128, 128);
  if (s.each() < 128 || mid < 3 * kCUs / 4) return Mx4Tile::t64x128;
  // 128 x 128 against 256 x 256, of which every CU takes whole rounds: a round
  // costs as much as 930 - K / 15 of the former, of which two share a CU.  us
  // at (M, N, K): (4096, 2560, 1024) 14.8 / 15.4, (4096, 2560, 4096) 36.9 /
  // 30.4, (4096, 4096, 1024) 18.4 / 17.9, (8192, 4096, 4096) 98 / 71; (512 rows
  // to each of 16 experts, N 2048, K 2048) 37 / 44.
  const int64_t big = up_to(s.tiles(256, 256), kCUs), less = s.K / 15 < 280 ? s.K / 15 : 280;
  return (mid + up_to(mid, 2 * kCUs) * 2 * kCUs) / 2 > big * (930 - less) ? Mx4Tile::t256x256 : Mx4Tile::t128x128;
}

}  // namespace bsq
