// Tiles of the ragged products on the device: how many there are, which
// segment a tile is of, and the order that they are taken in.
#pragma once

#include "common.h"
#include "lds.h"
#include "moe_index.h"

namespace bsq {

// The tiles of all segments (`total`), and the segment of the mt-th.  Every
// wave computes it alone: lane l sums the tiles of its share of the segments,
// a scan over the lanes finds the lane, and that lane's segments are walked.
template <int TM>
__device__ __forceinline__ int tiles_total(const Segments<TM>& seg, int lane, uint32_t& mine_before, uint32_t& mine) {
  mine = seg.lane_tiles(lane);
  uint32_t s = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  mine_before = s - mine;
  const uint32_t total = uint32_t(__builtin_amdgcn_readlane(int(s), 63)), limit = uint32_t(seg.limit());
  return scalar(int(total < limit ? total : limit));
}
template <int TM>
__device__ __forceinline__ Segment find_tile(const Segments<TM>& seg, int mt, uint32_t mine_before, uint32_t mine) {
  const uint64_t here = __ballot(Segments<TM>::has(mine_before, mine, mt));
  const int l = here ? __ffsll((unsigned long long)here) - 1 : 63;
  Segment s = seg.at(l, mt - __builtin_amdgcn_readlane(int(mine_before), l));
  s.e = __builtin_amdgcn_readfirstlane(s.e);
  s.row0 = __builtin_amdgcn_readfirstlane(s.row0);
  s.end = __builtin_amdgcn_readfirstlane(s.end);
  return s;
}

// Tile order: workgroups are dealt to the 8 XCDs round-robin by linear id,
// and each XCD has its own L2, so XCD x takes the x-th contiguous eighth of
// an order that walks bands of kBand tile rows column by column.  65536 rows
// over 32 experts, N 4096, K 2048: bands of 2, 4, 6, 8, 16 rows 662, 628, 610,
// 649, 673 us with an earlier output, of 4, 5, 6 rows 543, 531, 533 us with the
// present one; bands that end with the segments are no faster.
__device__ __forceinline__ void tile_order(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kBand = 5;
  const int T = tiles_m * tiles_n, per = T / 8;
  const int t = L < 8 * per ? (L % 8) * per + L / 8 : L;
  const int band = t / (kBand * tiles_n);
  const int rows = min(kBand, tiles_m - band * kBand);
  const int in = t - band * kBand * tiles_n;
  tm = band * kBand + in % rows;
  tn = in / rows;
}

}  // namespace bsq
