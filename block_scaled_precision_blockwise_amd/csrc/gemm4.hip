// Products with weights in microscaled 4 bits (e2m1 codes, E8M0 scales per 32):
//
//   out[r, n] = sum_k A[src(r), k] B[e, n, k]
//
// with A in e2m1, e4m3 or e5m2.  Dense: e is the product of the batch and
// src(r) = r.  Ragged: expert e's rows are the segment [offsets[e],
// offsets[e + 1]) of out, src(r) = rows[r] / k (or r); rows without a choice
// and rows past the last segment are written as zeros.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: both scales are applied in the matrix
// core, float32 accumulators.  A 16-byte chunk of packed codes is one block of
// 32 and one lane's operand, and two 4-bit operands take half the cycles of 8
// bits, so that a step of 128 bytes of each row is as much work for the matrix
// core, for LDS and for memory as one of the 8-bit products, and twice the
// contraction.  The MFMA's first operand is the B fragment, so that a lane's
// four results are four neighbours of one output row.
//
// K is any multiple of 32.  What the last step has not got is read from 16
// bytes of zeros, under scales of 1, so that no neighbour's code or NaN scale
// gets in.
#include "gemm4.h"
#include "lds.h"
#include "mx4_index.h"
#include "tiles.h"

#include <hip/hip_ext.h>
#include <type_traits>

namespace bsq {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __attribute__((aligned(16))) const uint8_t kZeros[16] = {};

struct Mx4Args {
  const uint8_t *A, *B, *SA, *SB;
  void* out;
  const int32_t *offsets, *rows;
  int64_t T, cap;
  int E, N, K, k;
  int bf16;
  int first;  // workgroup of this launch
};

// What a workgroup computes: output rows [m0, m_end) and columns from n0 of
// expert (or product) e.  `none`: no such expert, rows past the last segment.
struct Place4 {
  int e, m0, m_end, n0;
  bool none;
};

template <int FA>
struct View4 {  // FA: 0 e4m3, 1 e5m2, 4 e2m1
  const Mx4Args& p;
  __device__ __forceinline__ bool ragged() const { return p.offsets != nullptr; }
  __device__ __forceinline__ int64_t pitch_a() const { return FA == 4 ? p.K / 2 : p.K; }
  __device__ __forceinline__ int64_t pitch_b() const { return p.K / 2; }
  __device__ __forceinline__ int64_t pitch_s() const { return p.K / 32; }
  __device__ __forceinline__ const uint8_t* a(int e) const { return p.A + (ragged() ? 0 : int64_t(e) * p.T * pitch_a()); }
  __device__ __forceinline__ const uint8_t* sa(int e) const { return p.SA + (ragged() ? 0 : int64_t(e) * p.T * pitch_s()); }
  __device__ __forceinline__ const uint8_t* b(int e) const { return p.B + int64_t(e) * p.N * pitch_b(); }
  __device__ __forceinline__ const uint8_t* sb(int e) const { return p.SB + int64_t(e) * p.N * pitch_s(); }
  __device__ __forceinline__ int64_t row0(int e) const { return ragged() ? 0 : int64_t(e) * p.T; }  // of out
};

// What a lane knows of the tiles of all experts (or of the batch: `total` only).
struct Deal4 {
  int total;
  uint32_t before, mine;
};
template <int TM>
__device__ __forceinline__ Deal4 deal4(const Mx4Args& p, const int32_t* offsets, int lane) {
  Deal4 d{int((p.T + TM - 1) / TM) * p.E, 0, 0};
  if (p.offsets != nullptr) d.total = tiles_total(Segments<TM>{offsets, p.E, p.cap}, lane, d.before, d.mine);
  return d;
}

// The workgroup's tile `L`: along the columns first (few rows) or by
// tile_order.  `offsets`: the experts', or a copy of them.
template <int TM, int TN>
__device__ __forceinline__ bool find_place4(const Mx4Args& p, const int32_t* offsets, const Deal4& d, int L, bool along,
                                            Place4& t) {
  const int tiles_n = (p.N + TN - 1) / TN;
  int tm, tn;
  if (unsigned(L) >= unsigned(d.total) * unsigned(tiles_n)) return false;
  if (along) {
    tm = L / tiles_n;
    tn = L - tm * tiles_n;
  } else {
    tile_order(L, d.total, tiles_n, tm, tn);
  }
  if (p.offsets != nullptr) {
    const Segment s = find_tile(Segments<TM>{offsets, p.E, p.cap}, tm, d.before, d.mine);
    t.none = s.e >= p.E || p.T == 0;
    t.e = s.e < p.E ? s.e : 0;
    t.m0 = s.row0;
    t.m_end = s.end;
  } else {
    const int per = int((p.T + TM - 1) / TM);
    t.none = false;
    t.e = tm / per;
    t.m0 = (tm - t.e * per) * TM;
    t.m_end = int(p.T);
  }
  t.n0 = tn * TN;
  t.e = scalar(t.e);
  t.m0 = scalar(t.m0);
  t.m_end = scalar(t.m_end);
  t.n0 = scalar(t.n0);
  return true;
}

// The row of A of a tile's row r, -1 for none: the choice at the row, and the
// row of it.
__device__ __forceinline__ int choice4(const Mx4Args& p, const Place4& t, int r) {
  if (!row_in(t.m0, r, t.m_end) || t.none) return -1;
  return p.rows != nullptr ? p.rows[t.m0 + r] : t.m0 + r;
}
__device__ __forceinline__ int source4(const Mx4Args& p, int choice) {
  const int f = p.rows != nullptr && choice >= 0 ? choice / p.k : choice;
  return f >= p.T ? -1 : f;
}

__device__ __forceinline__ v8i wide(uint4 v) { return v8i{int(v.x), int(v.y), int(v.z), int(v.w), 0, 0, 0, 0}; }
__device__ __forceinline__ v8i wide(uint4 v, uint4 w) {
  return v8i{int(v.x), int(v.y), int(v.z), int(v.w), int(w.x), int(w.y), int(w.z), int(w.w)};
}

// acc += B fragment (e2m1) x A fragment (format FA), scales in the low bytes.
template <int FA>
__device__ __forceinline__ v4f mfma4(v8i b, v8i a, v4f acc, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc, 4, FA, 0, sb, 0, sa);
}

__device__ __forceinline__ void store4(const Mx4Args& p, int64_t at, v4f v) {
  if (p.bf16)
    __builtin_nontemporal_store(__builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4)),
                                reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + at));
  else
    __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(static_cast<float*>(p.out) + at));
}

// --------------------------------------------------------------- few rows --
// Tiles of 16 MB rows x 16 NB columns, where the weights' bytes are most of the
// work.  W waves share a tile's contraction, each with U chunks of 128 at a
// time, straight from memory to the operand registers, and their sums are
// joined through LDS in the waves' order.  U is 8 where every wave has as many,
// else 4.  Kernels in a replayed graph, weights from memory: 1 x 4096 x 14336 9.0
// us with 8, 10.5 with 4, x 4096 4.7 / 5.0; with less of the contraction to a
// wave (timed with 8 first) 8 x 2048 x 416 3.2 / 3.0, 1 x 8192 x 2880 6.0 / 5.8.
// Bound by the latency of a launch and of memory: one row of 8192 x 4096 6.1 us
// (17.8 MB, 2.9 TB/s), of 4096 x 4096 4.7 us, with weights that the caches hold
// 5.3 and 4.0.  Tiles of 64 x 64 this way are slower than through LDS (1024 x
// 1024 x 16384 40 us / 22): a load's 16 rows of 64 bytes are half lines.
template <int FA, int MB, int NB, int W, int U>
__global__ void __launch_bounds__(64 * W) k_mx4_few(Mx4Args p) {
  constexpr int TM = 16 * MB, TN = 16 * NB;
  constexpr int kPitch = TN + 4;  // of a row of sums, padded
  __shared__ __attribute__((aligned(16))) float red[W][TM][kPitch];
  __shared__ int src[TM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = scalar(tid >> 6);
  const View4<FA> view{p};
  Place4 t;
  if (!find_place4<TM, TN>(p, p.offsets, deal4<TM>(p, p.offsets, lane), p.first + int(blockIdx.x), true, t)) return;
  const int g = lane >> 4, r16 = lane & 15;
  bool any = false;
  const uint8_t *pa[MB], *psa[MB], *pb[NB], *psb[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int s = source4(p, choice4(p, t, 16 * i + r16)), row = s < 0 ? 0 : s;
    if (w == 0 && g == 0) src[16 * i + r16] = s;
    any |= s >= 0;
    pa[i] = view.a(t.e) + row * view.pitch_a();
    psa[i] = view.sa(t.e) + row * view.pitch_s();
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t row = min(t.n0 + 16 * j + r16, p.N - 1);
    pb[j] = view.b(t.e) + row * view.pitch_b();
    psb[j] = view.sb(t.e) + row * view.pitch_s();
  }
  const int nb = __ballot(any) ? p.K / 32 : 0;  // a tile without a choice is zeros
  v4f acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int c0 = w * U; 4 * c0 < nb; c0 += W * U) {
    uint4 b[U][NB], a[U][MB][FA == 4 ? 1 : 2];
    int sb[U][NB], sa[U][MB];
    const bool whole = 4 * (c0 + U) <= nb;
    if (whole) {
      // a row's scales 16 at a time: a load touches a line per row however little
      // it takes of it
      struct Scales {
        uint32_t v[U];
      };
      auto scales = [&](const uint8_t* row) {
        Scales s;
        __builtin_memcpy(&s, row + 4 * c0, 4 * U);
        return s;
      };
      Scales vb[NB], va[MB];
#pragma unroll
      for (int j = 0; j < NB; ++j) vb[j] = scales(psb[j]);
#pragma unroll
      for (int i = 0; i < MB; ++i) va[i] = scales(psa[i]);
      auto spread = [&](const Scales& s, int u) { return int(s.v[u] >> (8 * g)); };
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NB; ++j) b[u][j] = *reinterpret_cast<const uint4*>(pb[j] + 16 * (4 * (c0 + u) + g));
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if constexpr (FA == 4) {
            a[u][i][0] = *reinterpret_cast<const uint4*>(pa[i] + 16 * (4 * (c0 + u) + g));
          } else {
            // 8 bits: 16 elements of block g / 2 and 16 of block 2 + g / 2
#pragma unroll
            for (int h = 0; h < 2; ++h)
              a[u][i][h] = *reinterpret_cast<const uint4*>(pa[i] + 16 * (8 * (c0 + u) + 4 * h + g));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NB; ++j) sb[u][j] = spread(vb[j], u);
#pragma unroll
        for (int i = 0; i < MB; ++i) sa[u][i] = spread(va[i], u);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // past the end the last block's and chunk's, as zeros under scales of 1
        const int at = 4 * (c0 + u) + g, k0 = min(at, nb - 1);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          b[u][j] = *reinterpret_cast<const uint4*>(pb[j] + 16 * k0);
          sb[u][j] = at < nb ? psb[j][k0] : 127;
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          sa[u][i] = at < nb ? psa[i][k0] : 127;
#pragma unroll
          for (int h = 0; h < (FA == 4 ? 1 : 2); ++h) {
            const int n = FA == 4 ? nb : 2 * nb, c = FA == 4 ? at : 8 * (c0 + u) + 4 * h + g;
            const uint4 v = *reinterpret_cast<const uint4*>(pa[i] + 16 * min(c, n - 1));
            a[u][i][h] = c < n ? v : make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if constexpr (FA == 4) acc[j][i] = mfma4<FA>(wide(b[u][j]), wide(a[u][i][0]), acc[j][i], sb[u][j], sa[u][i]);
          else acc[j][i] = mfma4<FA>(wide(b[u][j]), wide(a[u][i][0], a[u][i][1]), acc[j][i], sb[u][j], sa[u][i]);
        }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) *reinterpret_cast<v4f*>(&red[w][16 * i + r16][16 * j + 4 * g]) = acc[j][i];
  __syncthreads();
  for (int q = tid; q < TM * TN / 4; q += 64 * W) {
    const int r = q / (TN / 4), c = 4 * (q % (TN / 4));
    if (!row_in(t.m0, r, t.m_end) || t.n0 + c >= p.N) continue;
    v4f v = *reinterpret_cast<const v4f*>(&red[0][r][c]);
#pragma unroll
    for (int x = 1; x < W; ++x) v += *reinterpret_cast<const v4f*>(&red[x][r][c]);
    if (src[r] < 0) v = v4f{0.f, 0.f, 0.f, 0.f};
    store4(p, (view.row0(t.e) + t.m0 + r) * p.N + t.n0 + c, v);
  }
}

// ------------------------------------------------------------------ tiles --
// WM x WN waves, each with MB x NB blocks of 16 x 16, K in steps of 128 bytes
// of A (256 elements of 4 bits, 128 of 8) through a ring of S LDS stages filled
// by direct loads.  A row's 16-byte chunks are XORed with half its number, so
// that the 16 rows of a fragment read fall on all 64 banks; B's rows of 64
// bytes (beside 8-bit A) lie two to a line.  A step waits for its own loads only.
//
// Scales of a row come 16 blocks, a unit of 2 steps of 4 bits or 4 of 8, at a
// time: a load of 64 rows' scales touches 64 lines however few bytes it takes
// of each.  They come as whole words: where K is no multiple of 128 a row's
// bytes start inside one, and one word more is read (AL 0).
//
// Where there are fewer tiles than CUs, KG groups of WM x WN waves share a
// tile's units (group i has i, i + KG, ..), each with a ring of its own, and
// their sums are joined through LDS in the groups' order.  A step has U parts.
//
// Measured: 1021 x 1792 x 2880, 8-bit A, 13.6 us (64 x 128, two groups); 1024 x
// 1024 x 16384 in 4 bits 21 us (64 x 64, two groups; one group 29), 600 ns for
// 512 of the contraction: more stages (3 to 5) or parts (1, 2) are within 0.5
// us of that, waves of 64 x 32 23.  64 rows x 4096 x 4096, held by the caches, 6.6
// us (32 x 64, two groups, two parts; one part 7.2), from memory 9.4.  8 tokens over 32 experts, N 4096, K 2048:
// 17 us, 5.3 TB/s (32 x 64).
template <int FA, int WM, int WN, int MB, int NB, int S, int KG, int U, int AL>
__global__ void __launch_bounds__(64 * WM * WN * KG, 1) k_mx4_tile(Mx4Args p) {
  constexpr int NW = WM * WN, TM = 16 * MB * WM, TN = 16 * NB * WN;
  constexpr int kPart = FA == 4 ? 256 : 128, kStep = U * kPart, kHalves = kPart / 128;
  constexpr int BA = 128, BB = kPart / 2;  // bytes of a row of a part of a step
  constexpr int RB = 1024 / BB;            // rows of B of a load
  constexpr int LA = TM / 8 / NW, LB = TN / RB / NW;
  static_assert(TM % (8 * NW) == 0 && TN % (RB * NW) == 0 && NW % 2 == 0, "whole loads of every wave");
  constexpr int SM = (TM + 63) / 64 * 64, SR = SM + TN;  // rows of scales
  static_assert(TN % 64 == 0, "scale rows by the 64");
  constexpr int kUnit = 512 / kStep;  // steps of 16 blocks
  static_assert(SR / 64 <= NW, "a wave has 64 rows of scales or none");
  constexpr int SU = (S - 1 + kUnit - 1) / kUnit + 1;  // units of scales that the steps under way are of
  constexpr int kPartBytes = TM * BA + TN * BB, kStage = U * kPartBytes;
  constexpr int kRowB = NB * 64 + 16;  // bytes of a staged output row of a wave, padded
  constexpr int kOut = NW * 16 * kRowB;
  constexpr int kJoin = (KG - 1) * NW * MB * NB * 1024;  // the other groups' accumulators
  constexpr int kMost = kOut > kJoin ? kOut : kJoin;
  constexpr int kAB = KG * S * kStage > kMost ? KG * S * kStage : kMost;
  __shared__ __attribute__((aligned(16))) uint8_t lds_ab[kAB];
  __shared__ __attribute__((aligned(16))) uint8_t lds_sc[KG][SU][SR * (AL ? 16 : 20)];
  __shared__ int src[TM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = scalar(tid >> 6) % NW, kg = scalar(tid >> 6) / NW;
  uint8_t* const lds = lds_ab + kg * S * kStage;
  uint8_t(*const lds_s)[SR * (AL ? 16 : 20)] = lds_sc[kg];
  const View4<FA> view{p};
  Place4 t;
  if (!find_place4<TM, TN>(p, p.offsets, deal4<TM>(p, p.offsets, lane), p.first + int(blockIdx.x), false, t)) return;
  int any = 0;
  for (int r = tid; r < TM; r += 64 * NW * KG) {
    src[r] = source4(p, choice4(p, t, r));
    any |= src[r] >= 0;
  }
  // a tile without a choice is zeros (a plan's alignment leaves such tiles)
  const int all = __syncthreads_or(any) ? (p.K + kStep - 1) / kStep : 0;
  // units of the tile and of the group, steps of the group
  const int units = (all + kUnit - 1) / kUnit, mine = (units - kg + KG - 1) / KG;
  const int nk = mine * kUnit - ((units - 1) % KG == kg ? units * kUnit - all : 0);
  auto global = [&](int i) { return (KG * (i / kUnit) + kg) * kUnit + i % kUnit; };  // step of the group's i-th

  // ---- loads: lane i of a load of A fills row i / 8, chunk place i % 8
  const int lrow = lane >> 3, ca = 16 * ((lane & 7) ^ (4 * (w & 1) + (lrow >> 1)));
  // of B: the same, or (64-byte rows) line i / 8, place i % 8: row 2 (i / 8) +
  // (i % 8) / 4, chunk i % 4 XORed with half the line's number
  const int brow = BB == 128 ? lrow : 2 * lrow + ((lane >> 2) & 1);
  const int cb = BB == 128 ? ca : 16 * ((lane & 3) ^ ((lrow >> 1) & 3));
  const uint8_t *pa[LA], *pb[LB];
#pragma unroll
  for (int s = 0; s < LA; ++s)
    pa[s] = view.a(t.e) + int64_t(max(src[8 * (w + NW * s) + lrow], 0)) * view.pitch_a() + ca;
#pragma unroll
  for (int s = 0; s < LB; ++s)
    pb[s] = view.b(t.e) + int64_t(min(t.n0 + RB * (w + NW * s) + brow, p.N - 1)) * view.pitch_b() + cb;
  const uint32_t la = lds_of(lds + 1024 * w), lb = lds_of(lds + TM * BA + 1024 * w);
  const int64_t last = int64_t(all - 1) * U * BA, last_b = int64_t(all - 1) * U * BB;
  const bool part = p.K % kStep != 0;
  // scales: wave w has rows 64 w .. of A's and then B's
  const int64_t sp = view.pitch_s();
  const uint64_t sa0 = reinterpret_cast<uint64_t>(view.sa(t.e));
  const int bm = int(sa0 & 3);  // a batch's scales need not start a word
  auto a_row = [&](int r) { return max(src[r], 0); };
  auto b_row = [&](int r) { return min(t.n0 + r, p.N - 1); };
  const bool has = w < SR / 64;
  const int srow = 64 * w + lane;
  const i32x4 rs = w < SM / 64 ? rsrc(reinterpret_cast<const uint8_t*>(sa0 - bm), (bm + p.T * sp + 3) & ~int64_t(3))
                               : rsrc(view.sb(t.e), p.N * sp);
  const uint32_t so = (srow < SM ? uint32_t(bm + a_row(min(srow, TM - 1)) * sp) : uint32_t(b_row(srow - SM) * sp)) & ~3u;
  const uint32_t ls = lds_of(&lds_s[0][64 * w * 16]), ls4 = lds_of(&lds_s[0][SR * 16 + 64 * w * 4]);
  constexpr int kLoads = U * (LA + LB), kScales = AL ? 1 : 2;  // of a step, of a unit
  const uint8_t* const zeros = kZeros;
  auto load = [&](int i, int st) {  // the group's i-th step
    const int ks = global(i);
    const uint32_t at = uint32_t(st * kStage);
    if (has && i % kUnit == 0) {
      const uint32_t from = so + 16u * uint32_t(ks / kUnit), to = uint32_t(i / kUnit % SU * SR * (AL ? 16 : 20));
      dma16(rs, from, ls + to);
      if (!AL) dma4(rs, from + 16u, ls4 + to);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t to = at + uint32_t(u * kPartBytes);
      if (part && ks == all - 1) {  // zeros where the last step has not got the lane's chunk
        const bool past_a = last + u * BA + ca >= view.pitch_a(), past_b = last_b + u * BB + cb >= view.pitch_b();
#pragma unroll
        for (int s = 0; s < LA; ++s) dma16(past_a ? zeros : pa[s] + last + u * BA, la + to + uint32_t(1024 * NW * s));
#pragma unroll
        for (int s = 0; s < LB; ++s) dma16(past_b ? zeros : pb[s] + last_b + u * BB, lb + to + uint32_t(1024 * NW * s));
      } else {
#pragma unroll
        for (int s = 0; s < LA; ++s) dma16(pa[s] + (int64_t(ks) * U + u) * BA, la + to + uint32_t(1024 * NW * s));
#pragma unroll
        for (int s = 0; s < LB; ++s) dma16(pb[s] + (int64_t(ks) * U + u) * BB, lb + to + uint32_t(1024 * NW * s));
      }
    }
  };

  const int wm = w % WM, wn = w / WM, g = lane >> 4, r16 = lane & 15;
  const int x8 = r16 >> 1;  // what a row's chunks are XORed with
  // the byte of a unit's scales that the lane's block of the first MFMA has
  int ma[MB], mb = g;
#pragma unroll
  for (int i = 0; i < MB; ++i)
    ma[i] = g + (AL ? 0 : int((unsigned(bm) + unsigned(a_row(16 * MB * wm + 16 * i + r16)) * unsigned(sp)) & 3u));
  if (!AL) mb += int((unsigned(b_row(16 * NB * wn + r16)) * unsigned(sp)) & 3u);
  v4f acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int i = 0; i < min(nk, S - 1); ++i) load(i, i);

  int st = 0;
  uint32_t qa[4][MB], qb[4][NB];  // scales of the unit's MFMAs, in the low byte
  // One step, the `at`-th of unit u.
  auto step = [&](int u, int at) {
    const int i = u * kUnit + at;
    // S - 2 steps (and what scales come with them) stay under way; near the end,
    // where fewer are, all are waited for
    // (units that start among the S - 2 steps: `starts`)
    const int starts = (at + S - 2) / kUnit;
    static_assert((kUnit - 1 + S - 2) / kUnit <= 2, "at most two");
    if (i + S - 2 >= nk) __builtin_amdgcn_s_waitcnt(vmcnt(0));
    else if (has && starts == 2) __builtin_amdgcn_s_waitcnt(vmcnt((S - 2) * kLoads + 2 * kScales));
    else if (has && starts == 1) __builtin_amdgcn_s_waitcnt(vmcnt((S - 2) * kLoads + kScales));
    else __builtin_amdgcn_s_waitcnt(vmcnt((S - 2) * kLoads));
    barrier();
    if (i >= nk) return;  // other groups' steps
    // past the barrier nobody reads the stage before this one
    if (i + S - 1 < nk) load(i + S - 1, st == 0 ? S - 1 : st - 1);
    if (at == 0) {
      const uint8_t* const ss = lds_s[u % SU];
      auto scales = [&](int row, int byte, uint32_t (&q)[4]) {
        const uint4 v = *reinterpret_cast<const uint4*>(ss + 16 * row);
        uint32_t x[5] = {v.x, v.y, v.z, v.w, 0u};
        if (!AL) x[4] = *reinterpret_cast<const uint32_t*>(ss + 16 * SR + 4 * row);
#pragma unroll
        for (int d = 0; d < 4; ++d) q[d] = (!AL && byte >= 4 ? x[d + 1] : x[d]) >> (8 * (byte & 3));
      };
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        uint32_t q[4];
        scales(16 * MB * wm + 16 * i + r16, ma[i], q);
#pragma unroll
        for (int d = 0; d < 4; ++d) qa[d][i] = q[d];
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        uint32_t q[4];
        scales(SM + 16 * NB * wn + 16 * j + r16, mb, q);
#pragma unroll
        for (int d = 0; d < 4; ++d) qb[d][j] = q[d];
      }
      const int left = p.K / 32 - (KG * u + kg) * 16;  // blocks from the unit on
      if (left < 16) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const bool past = 4 * d + g >= left;
#pragma unroll
          for (int i = 0; i < MB; ++i) qa[d][i] = past ? 127u : qa[d][i];
#pragma unroll
          for (int j = 0; j < NB; ++j) qb[d][j] = past ? 127u : qb[d][j];
        }
      }
    }
    auto chunk = [&](const uint8_t* tile, int row, int c) {  // of a 128-byte row
      return *reinterpret_cast<const uint4*>(tile + row * 128 + 16 * (c ^ x8));
    };
    auto bfrag = [&](const uint8_t* tb, int h, int j) {
      const int row = 16 * NB * wn + 16 * j + r16;
      if constexpr (BB == 128) return wide(chunk(tb, row, 4 * h + g));
      else return wide(*reinterpret_cast<const uint4*>(tb + (row >> 1) * 128 + 64 * (row & 1) + 16 * (g ^ ((row >> 2) & 3))));
    };
#pragma unroll
    for (int c = 0; c < U * kHalves; ++c) {  // chunks of 128 of the contraction
      const int h = c % kHalves, n = U * kHalves * at + c;
      const uint8_t* ta = lds + st * kStage + c / kHalves * kPartBytes;
      const uint8_t* tb = ta + TM * BA;
      v8i fa[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int row = 16 * MB * wm + 16 * i + r16;
        if constexpr (FA == 4) fa[i] = wide(chunk(ta, row, 4 * h + g));
        else fa[i] = wide(chunk(ta, row, g), chunk(ta, row, 4 + g));
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const v8i fb = bfrag(tb, h, j);
#pragma unroll
        for (int i = 0; i < MB; ++i)
          acc[j][i] = mfma4<FA>(fb, fa[i], acc[j][i], int(qb[n][j]), int(qa[n][i]));
      }
    }
    st = st == S - 1 ? 0 : st + 1;
  };
  for (int u = 0; u < (units + KG - 1) / KG; ++u) {
#pragma unroll
    for (int at = 0; at < kUnit; ++at) step(u, at);
  }

  if constexpr (KG > 1) {
    v4f* const join = reinterpret_cast<v4f*>(lds_ab) + 64 * MB * NB * w + lane;
    __syncthreads();
    if (kg > 0) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) join[64 * MB * NB * NW * (kg - 1) + 64 * (MB * j + i)] = acc[j][i];
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int o = 0; o < KG - 1; ++o)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int i = 0; i < MB; ++i) acc[j][i] += join[64 * MB * NB * NW * o + 64 * (MB * j + i)];
    }
  }

  // ---- out: 16 rows of the wave at a time through LDS, so that a store
  // instruction writes whole rows of the wave's columns
  uint8_t* const stg = lds_ab + w * 16 * kRowB;
  constexpr int LPR = 4 * NB, RPI = 64 / LPR;
  static_assert(64 % LPR == 0, "whole rows per instruction");
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<v4f*>(stg + r16 * kRowB + (16 * j + 4 * g) * 4) = acc[j][i];
    }
    __syncthreads();
    if (kg > 0) continue;
#pragma unroll
    for (int q = 0; q < 16 / RPI; ++q) {
      const int rr = RPI * q + lane / LPR, cc = 4 * (lane % LPR);
      const int tr = 16 * MB * wm + 16 * i + rr, n = t.n0 + 16 * NB * wn + cc;
      v4f v = *reinterpret_cast<const v4f*>(stg + rr * kRowB + cc * 4);
      if (src[tr] < 0) v = v4f{0.f, 0.f, 0.f, 0.f};
      if (row_in(t.m0, tr, t.m_end) && n < p.N) store4(p, (view.row0(t.e) + t.m0 + tr) * p.N + n, v);
    }
  }
}

// -------------------------------------------------------------- big tiles --
// 256 x 256 by four waves of 128 x 128, one wave per SIMD: a step's LDS reads
// are 128 KiB for 512 4-bit MFMAs of 16 cycles on four SIMDs, and the
// accumulators of a wave fill the 256 accumulation registers.  With nothing
// else to run on its SIMD a wave may never wait, so it goes through a step in
// four phases, one for each pairing of the halves of its A and B fragments (A0
// B0, A0 B1, A1 B1, A1 B0), and reads beside each the half that a later phase
// needs: B1 and A1 of this step, then A0 and B0 of the next (B0 fragment by
// fragment, as its last MFMAs pass).  The reads of a stage end in its second
// phase: the step's one barrier is there, the loads of the step after next
// follow it, and have until the next barrier to land.
//
// Scales of 16 blocks of a row (a group of 2 steps of 4 bits, 4 of 8) go
// through registers, so that they may start at any byte: what the contraction
// has not got becomes 1, and the 4 x 4 bytes are transposed, so that a lane's
// one word holds its block of each of four MFMAs.
//
// A workgroup goes through the tiles blockIdx.x + gridDim.x i.  Between two of
// them come the loads of the next one's first two steps, then the output of the
// last one, from the accumulators to memory without LDS (lanes exchange halves
// until each holds 16 neighbouring bytes of a row).  Where the tile is whole the
// number of its stores is known, and they are left under way: the waits for the
// next tile's first steps count them out (360 us where waiting for them took
// 391, the experts of 65536 rows below).  The search for a tile is made of a copy
// of the offsets in LDS, so that it waits for no load.
//
// Measured: 16384 x 8192 x 4096 in 4 bits 263 us, 4.2 PFLOP/s; 65536 rows over
// 32 experts, N 4096, K 2048, 360 us, 3.1; 8192 x 4096 x 4096 with e4m3 106 us,
// 2.6.  Pure MFMAs on random codes reach 6.6-6.9 PFLOP/s (9.0 on zeros: the clock
// gives way), e2m1 times e4m3 4.3 (4.9).  Of the 263 us the loads are 32,
// the stores 30, the LDS reads 10; two wait states in front of every MFMA and of
// every load's m0 were 25 more.

// 16 bytes from any address before `end`, which has 16 in front of it: the last
// 16 where fewer are left.
__device__ __forceinline__ uint4 scales16(const uint8_t* p, const uint8_t* end) {
  uint4 v;
  __builtin_memcpy(&v, p + 16 <= end ? p : end - 16, 16);
  return v;
}
// The 4 x 4 bytes transposed.  Where a row ends (n < 16), the bytes that are
// there are brought to the front by `skip` and the rest becomes 0x7F.
__device__ __forceinline__ uint4 turned(uint4 v, int n, int skip) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (n < 16) {
    uint32_t x[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t lo = 0u, hi = 0u;  // the words that word d of the shifted bytes spans
#pragma unroll
      for (int i = d; i < 4; ++i) {
        if (i == d + (skip >> 2)) lo = w[i];
        if (i == d + (skip >> 2) + 1) hi = w[i];
      }
      x[d] = __builtin_amdgcn_alignbyte(hi, lo, uint32_t(skip & 3));
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int have = min(max(n - 4 * d, 0), 4);
      const uint32_t keep = uint32_t((uint64_t(1) << (8 * have)) - 1);
      w[d] = (x[d] & keep) | (0x7F7F7F7Fu & ~keep);
    }
  }
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  return make_uint4(__builtin_amdgcn_perm(c, a, 0x05040100u), __builtin_amdgcn_perm(c, a, 0x07060302u),
                    __builtin_amdgcn_perm(d, b, 0x05040100u), __builtin_amdgcn_perm(d, b, 0x07060302u));
}

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kMaxEnds = 1025;  // of the experts' segments

// acc += b x a in inline asm, for its place among the loads and reads (the
// compiler moves the builtin past all of them) and for accumulation registers.
// HH: the byte of both scale words.  Its operands come from LDS reads, which
// the compiler waits for; the scale words may come from vector instructions,
// two wait states after which are the caller's.  Back to back on one
// accumulator needs none.
#define BSQ_MFMA4(SEL, FMT) "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4" FMT
#define BSQ_MFMA4_FA(SEL, ...)                                   \
  do {                                                           \
    if constexpr (FA == 4) __VA_ARGS__(BSQ_MFMA4(SEL, " blgp:4"), a_lo); \
    else if constexpr (FA == 1) __VA_ARGS__(BSQ_MFMA4(SEL, " blgp:1"), a); \
    else __VA_ARGS__(BSQ_MFMA4(SEL, ""), a);                     \
  } while (0)
#define BSQ_MFMA4_HH(...)                                                                  \
  do {                                                                                     \
    if constexpr (HH == 0) BSQ_MFMA4_FA("op_sel_hi:[0,0,0]", __VA_ARGS__);                 \
    else if constexpr (HH == 1) BSQ_MFMA4_FA("op_sel:[1,1,0] op_sel_hi:[0,0,0]", __VA_ARGS__); \
    else if constexpr (HH == 2) BSQ_MFMA4_FA("op_sel_hi:[1,1,0]", __VA_ARGS__);            \
    else BSQ_MFMA4_FA("op_sel:[1,1,0] op_sel_hi:[1,1,0]", __VA_ARGS__);                    \
  } while (0)
template <int FA, int HH>
__device__ __forceinline__ void mfma_at(v4f& acc, v4i b, const v8i& a, int sb, int sa) {
  const v4i a_lo = __builtin_shufflevector(a, a, 0, 1, 2, 3);
#define BSQ_PLAIN(TEXT, A) asm volatile(TEXT : "+a"(acc) : "v"(b), "v"(A), "v"(sb), "v"(sa))
  BSQ_MFMA4_HH(BSQ_PLAIN);
#undef BSQ_PLAIN
}
// The same, and a load of 16 bytes per lane into LDS behind it (see dma16): the
// MFMA is the wait state between m0 and the load.
template <int FA, int HH>
__device__ __forceinline__ void mfma_at(v4f& acc, v4i b, const v8i& a, int sb, int sa, const uint8_t* base, uint32_t off,
                                        uint32_t lds, int at) {
  const v4i a_lo = __builtin_shufflevector(a, a, 0, 1, 2, 3);
#define BSQ_LOADS(TEXT, A)                                                                           \
  asm volatile("s_add_u32 m0, %5, %8\n\t" TEXT "\n\tglobal_load_lds_dwordx4 %6, %7"                 \
               : "+a"(acc)                                                                           \
               : "v"(b), "v"(A), "v"(sb), "v"(sa), "s"(lds), "v"(off), "s"(base), "i"(at)            \
               : "memory", "scc")
  BSQ_MFMA4_HH(BSQ_LOADS);
#undef BSQ_LOADS
}
#undef BSQ_MFMA4_HH
#undef BSQ_MFMA4_FA
#undef BSQ_MFMA4

template <int FA, int OUT_BF16>
__global__ void __launch_bounds__(256, 1) k_mx4_big(Mx4Args p) {
  constexpr int TM = 256, TN = 256, NW = 4;
  constexpr int kStep = FA == 4 ? 256 : 128, kHalves = kStep / 128, kGroup = 512 / kStep;  // steps of 16 blocks
  constexpr int BA = 128, BB = kStep / 2, RB = 1024 / BB, LB = TN / RB / NW;  // loads of B per wave and step
  constexpr int kStage = TM * BA + TN * BB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds_s[2 * (TM + TN) * 16];
  __shared__ int src[2][TM];
  __shared__ int32_t ends[kMaxEnds];
  // stores of a whole tile by a wave; what vmcnt can count of them
  constexpr int kStores = OUT_BF16 ? 32 : 63;

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = scalar(tid >> 6);
  const View4<FA> view{p};
  const int nb = p.K / 32, all = (p.K + kStep - 1) / kStep;
  const bool part = p.K % kStep != 0;

  // ---- loads: 8 slices of 8 rows of A per wave (and of B, or 4 of 16 rows of
  // 64 bytes); lane i fills the i-th 16 bytes of a slice with the chunk that
  // the swizzle keeps there (see k_mx4_tile).  32-bit offsets from a base that
  // moves on by a step (the launcher sends what they do not reach elsewhere).
  const int lrow = lane >> 3, ca = 16 * ((lane & 7) ^ (4 * (w & 1) + (lrow >> 1)));
  const int brow = BB == 128 ? lrow : 2 * lrow + ((lane >> 2) & 1);
  const int cb = BB == 128 ? ca : 16 * ((lane & 3) ^ ((lrow >> 1) & 3));
  // whether the last step has not got the lane's chunk: it loads the row's
  // first of that step instead, and puts zeros over it
  const bool past_a = part && int64_t(all - 1) * BA + ca >= view.pitch_a();
  const bool past_b = part && int64_t(all - 1) * BB + cb >= view.pitch_b();
  const uint8_t *pa, *pb;
  uint32_t off[8 + LB];
  const uint32_t lbase = lds_of(lds + 1024 * w);
  uint32_t to = lbase;  // stage that is loaded
  auto last_step = [&] {  // before the loads of a tile's last step
#pragma unroll
    for (int s = 0; s < 8 + LB; ++s) off[s] -= s < 8 ? (past_a ? uint32_t(ca) : 0u) : (past_b ? uint32_t(cb) : 0u);
  };
  auto place = [&](int s) { return s < 8 ? 1024 * NW * s : TM * BA + 1024 * NW * (s - 8); };  // in the stage
  auto load = [&](int s, uint32_t to) { dma16(s < 8 ? pa : pb, off[s], to, place(s)); };
  auto loaded = [&] {  // a whole step
    pa += BA;
    pb += BB;
    to = 2 * lbase + kStage - to;
  };
  // Zeros over the chunks that the last step, in the stage from `stage` bytes
  // on, has not got; its loads have landed.
  auto blank = [&](int stage) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint8_t* const at = lds + stage + 1024 * w + 16 * lane;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (past_a) *reinterpret_cast<uint4*>(at + 1024 * NW * s) = zero;
#pragma unroll
    for (int s = 0; s < LB; ++s)
      if (past_b) *reinterpret_cast<uint4*>(at + TM * BA + 1024 * NW * s) = zero;
  };
  // scales: thread t has row t of A and of B, 16 blocks at a time
  const uint8_t *sa_row, *sb_row, *sa_end, *sb_end;
  uint4 va, vb;
  auto load_scales = [&](int q) {
    va = scales16(sa_row + 16 * q, sa_end);
    vb = scales16(sb_row + 16 * q, sb_end);
  };
  auto put_scales = [&](int q) {
    uint8_t* const at = lds_s + (q & 1) * (TM + TN) * 16 + 16 * tid;
    auto skip = [&](const uint8_t* row, const uint8_t* end) { return max(int(row + 16 * q + 16 - end), 0); };
    *reinterpret_cast<uint4*>(at) = turned(va, nb - 16 * q, skip(sa_row, sa_end));
    *reinterpret_cast<uint4*>(at + TM * 16) = turned(vb, nb - 16 * q, skip(sb_row, sb_end));
  };
  // Addresses of tile t, whose rows of A are in src[buf], and its first scales.
  auto begin = [&](const Place4& t, int buf) {
    if (t.none) return;
    // rows of their own are near the tile's first; gathered ones anywhere
    const int near = p.rows != nullptr ? 0 : min(t.m0, int(p.T) - 1);
    auto a_row = [&](int r) { return max(src[buf][r], near) - near; };
    pa = scalar(view.a(t.e) + near * view.pitch_a());
    pb = scalar(view.b(t.e) + int64_t(t.n0) * view.pitch_b());
#pragma unroll
    for (int s = 0; s < 8; ++s)
      off[s] = uint32_t(a_row(8 * (w + NW * s) + lrow)) * uint32_t(view.pitch_a()) + uint32_t(ca);
#pragma unroll
    for (int s = 0; s < LB; ++s)
      off[8 + s] = uint32_t(min(RB * (w + NW * s) + brow, p.N - 1 - t.n0)) * uint32_t(view.pitch_b()) + uint32_t(cb);
    const int64_t sp = view.pitch_s();
    sa_row = view.sa(t.e) + (int64_t(a_row(tid)) + near) * sp;
    sb_row = view.sb(t.e) + int64_t(min(t.n0 + tid, p.N - 1)) * sp;
    sa_end = view.sa(t.e) + p.T * sp;
    sb_end = view.sb(t.e) + p.N * sp;
    to = lbase;
    load_scales(0);
  };
  // The loads of a tile's first two steps.
  auto preload = [&](int nk) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (nk <= q) return;
      const uint32_t stage = uint32_t(scalar(int(lbase + (q ? kStage : 0))));
      if (part && q == nk - 1) last_step();
#pragma unroll
      for (int s = 0; s < 8 + LB; ++s) load(s, stage);
      loaded();
    }
  };

  const int wm = w & 1, wn = w >> 1, g = lane >> 4, r16 = lane & 15;
  const int ra = (128 * wm + r16) * BA, rb = TM * BA + (128 * wn + r16) * BB;
  const int x8 = r16 >> 1;
  // of the stage that is read: where a row's two chunks are
  const int oa0 = ra + 16 * (g ^ x8), oa1 = ra + 16 * ((4 + g) ^ x8);
  const int ob0 = BB == 128 ? rb + 16 * (g ^ x8)
                            : TM * BA + (64 * wn + x8) * 128 + 64 * (r16 & 1) + 16 * (g ^ ((r16 >> 2) & 3));
  const int ob1 = rb + 16 * ((4 + g) ^ x8);
  const int ssa = (128 * wm + r16) * 16 + 4 * g, ssb = (TM + 128 * wn + r16) * 16 + 4 * g;
  v4f acc[8][8];  // [column block][row block]
  v8i fa[8];
  v4i fb[8][kHalves];
  int qa[8], qb[8];
  int o = 0;  // stage that is read
  auto a_part = [&](int f, int h) {  // 16 bytes of a fragment
    const uint4 v = *reinterpret_cast<const uint4*>(lds + o + (h ? oa1 : oa0) + 16 * f * BA);
    fa[f][4 * h] = int(v.x);
    fa[f][4 * h + 1] = int(v.y);
    fa[f][4 * h + 2] = int(v.z);
    fa[f][4 * h + 3] = int(v.w);
  };
  auto b_part = [&](int f, int h) {
    const uint4 v = *reinterpret_cast<const uint4*>(lds + o + (h ? ob1 : ob0) + 16 * f * BB);
    fb[f][h] = v4i{int(v.x), int(v.y), int(v.z), int(v.w)};
  };
  auto scale_a = [&](int q, int f) -> int {
    return *reinterpret_cast<const int*>(lds_s + (q & 1) * (TM + TN) * 16 + ssa + 16 * 16 * f);
  };
  auto scale_b = [&](int q, int f) -> int {
    return *reinterpret_cast<const int*>(lds_s + (q & 1) * (TM + TN) * 16 + ssb + 16 * 16 * f);
  };
  // Nothing, but no use of an accumulator moves past it.
  auto settle = [&] {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) asm volatile("" : "+a"(acc[j][i]));
  };
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  // The MFMAs of the halves j0 of B and i0 of A, column by column, two blocks
  // at a time.  P: which bytes of the scale words; the first MFMA of the x-th
  // two brings load `first` + x where there is one before `end`; `beside(x)`
  // comes after it.
  uint32_t fill = lbase;  // stage that the loads go to
  auto phase = [&](int j0, int i0, auto at, int first, int end, auto&& beside) {
    constexpr int H = kHalves * decltype(at)::value;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = j0 + x / 2, i = i0 + 2 * (x & 1), s = first + x;
      if (s < end)
        mfma_at<FA, H>(acc[j][i], fb[j][0], fa[i], qb[j], qa[i], s < 8 ? pa : pb, off[s], fill, place(s));
      else
        mfma_at<FA, H>(acc[j][i], fb[j][0], fa[i], qb[j], qa[i]);
      beside(x);
      mfma_at<FA, H>(acc[j][i + 1], fb[j][0], fa[i + 1], qb[j], qa[i + 1]);
      if constexpr (kHalves == 2) {
        const v8i a0 = __builtin_shufflevector(fa[i], fa[i], 4, 5, 6, 7, 4, 5, 6, 7);
        const v8i a1 = __builtin_shufflevector(fa[i + 1], fa[i + 1], 4, 5, 6, 7, 4, 5, 6, 7);
        mfma_at<FA, H + 1>(acc[j][i], fb[j][kHalves - 1], a0, qb[j], qa[i]);
        mfma_at<FA, H + 1>(acc[j][i + 1], fb[j][kHalves - 1], a1, qb[j], qa[i + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  bool stored = false;  // the last tile's stores may still be under way
  // Step ks.  LOADS: the step after next follows it, and is loaded.  TURN: what
  // becomes of the scale words for the next step.  0: they stay, and its bytes
  // are the next (4 bits: the first step of a group); 1: another group's are
  // read; 2: its group's are read and shifted.  P: the bytes of this step.
  auto step = [&](int ks, int nk, auto loads, auto turn, auto at) {
    constexpr bool LOADS = decltype(loads)::value;
    constexpr int TURN = decltype(turn)::value;
    const int q = (ks + 1) / kGroup, next_at = (ks + 1) % kGroup;  // of the next step
    constexpr int kEnd = LOADS ? 8 + LB : 0;
    phase(0, 0, at, 0, 0, [&](int x) {
      if (x % 2 < kHalves) b_part(4 + x / 2, x & 1);
    });
    phase(4, 0, at, 0, 0, [&](int x) { a_part(4 + x / 2, x & 1); });
    if (ks == 0 && stored) __builtin_amdgcn_s_waitcnt(vmcnt(kStores));
    else __builtin_amdgcn_s_waitcnt(vmcnt(0));
    if (part && ks + 1 == nk - 1) blank(o ^ kStage);
    if (TURN && next_at == 0 && ks + 1 < nk) put_scales(q);
    barrier();
    if (LOADS && TURN != 1 && next_at == kGroup - 1) load_scales(q + 1);
    o ^= kStage;
    fill = uint32_t(scalar(int(to)));
    if (LOADS && part && ks + 2 == nk - 1) last_step();
    int next[16];  // scales of the next step
    phase(4, 4, at, 0, kEnd < 8 ? kEnd : 8, [&](int x) {
      a_part(x / 2, x & 1);
      if (TURN) next[x] = scale_a(q, x);
    });
    // fragment f of B0 is free after its last MFMA
    phase(0, 4, at, 8, kEnd, [&](int x) {
      if (x >= 2 && x % 2 < kHalves) b_part(x / 2 - 1, x & 1);
      if (TURN) next[8 + x] = scale_b(q, x);
    });
#pragma unroll
    for (int h = 0; h < kHalves; ++h) b_part(3, h);
    // in inline asm, so that they stay behind the MFMAs
    if constexpr (TURN) {
      const int bits = TURN == 1 ? 0 : 8 * kHalves * next_at;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        asm volatile("v_lshrrev_b32 %0, %2, %1" : "=v"(qa[i]) : "v"(next[i]), "s"(bits));
        asm volatile("v_lshrrev_b32 %0, %2, %1" : "=v"(qb[i]) : "v"(next[8 + i]), "s"(bits));
      }
      asm volatile("s_nop 1");
    }
    if (LOADS) loaded();
  };
  // ---- out: lane (g, r16) has columns 4 g .. 4 g + 3 of row r16 of each
  // block.  bfloat16: of two blocks' eight, halves of the wave and then rows
  // of 16 lanes change places until it has columns 8 g .. 8 g + 7 of the 32;
  // then neighbouring rows trade one pair of blocks each, so that a store
  // writes whole 128-byte lines.
  auto output = [&](const Place4& t, int buf, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;  // every row and column is there
    constexpr int kElem = OUT_BF16 ? 2 : 4;
    const int64_t pitch = int64_t(p.N) * kElem;
    const int n0 = t.n0 + 128 * wn, left = p.N - n0;  // columns of the wave
    uint8_t* at = static_cast<uint8_t*>(p.out) + view.row0(t.e) * pitch + byte_at(t.m0, 128 * wm, pitch, n0, kElem);
    const bool odd = r16 & 1;
    uint8_t* const pair = at + (r16 & 14) * pitch + (odd ? 64 : 0) + 16 * g;
    at += r16 * pitch + 16 * g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int tr = 128 * wm + 16 * i + r16;
      const bool none = src[buf][tr] < 0, in = row_in(t.m0, tr, t.m_end);
      if constexpr (OUT_BF16) {
        const bool even_in = row_in(t.m0, tr & ~1, t.m_end), odd_in = row_in(t.m0, tr | 1, t.m_end);
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // 64 columns
          uint32_t v[2][4];            // 8 columns of 32, twice
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = 4 * q + 2 * h;
            const u32x2 x = __builtin_bit_cast(u32x2, __builtin_convertvector(acc[j][i], bf16x4));  // to nearest even
            const u32x2 y = __builtin_bit_cast(u32x2, __builtin_convertvector(acc[j + 1][i], bf16x4));
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              const auto a = __builtin_amdgcn_permlane32_swap(x[d], y[d], false, false);
              const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[1], false, false);
              v[h][d] = none ? 0u : uint32_t(b[0]);
              v[h][2 + d] = none ? 0u : uint32_t(b[1]);
            }
          }
          u32x4_t even_row, odd_row;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint32_t got = uint32_t(__builtin_amdgcn_mov_dpp(int(odd ? v[0][d] : v[1][d]), 0xB1, 0xF, 0xF, true));
            even_row[d] = odd ? got : v[0][d];
            odd_row[d] = odd ? v[1][d] : got;
          }
          if (kWhole || 64 * q + (odd ? 32 : 0) + 8 * g < left) {
            uint8_t* const to = pair + 16 * i * pitch + 128 * q;
            if (kWhole || even_in) __builtin_nontemporal_store(even_row, reinterpret_cast<u32x4_t*>(to));
            if (kWhole || odd_in) __builtin_nontemporal_store(odd_row, reinterpret_cast<u32x4_t*>(to + pitch));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v4f v;  // one at a time out of the accumulation registers
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            float x;
            asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(x) : "a"(acc[j][i][d]));
            v[d] = none ? 0.f : x;
          }
          if (kWhole || (in && 16 * j + 4 * g < left))
            __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(at + 16 * i * pitch + 64 * j));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The wait for a tile's first step, whose loads were followed by `kept` stores
  // at least.
  auto arrive = [&](int nk, int kept) {
    if (nk > 0) put_scales(0);
    if (kept) __builtin_amdgcn_s_waitcnt(vmcnt(kStores));
    else __builtin_amdgcn_s_waitcnt(vmcnt(0));
    if (part && nk == 1) blank(0);
  };

  const Deal4 deal = deal4<TM>(p, p.offsets, lane);
  if (p.offsets != nullptr) {
    for (int i = tid; i <= p.E; i += 256) ends[i] = p.offsets[i];
    __syncthreads();
  }
  Place4 cur, next{};
  int L = blockIdx.x, buf = 0;
  if (!find_place4<TM, TN>(p, ends, deal, L, false, cur)) return;
  src[0][tid] = source4(p, choice4(p, cur, tid));
  __syncthreads();
  begin(cur, 0);
  int nk = cur.none ? 0 : all;
  preload(nk);
  arrive(nk, 0);
  clear();
  for (;;) {
    // the search for the next tile reads LDS only, and the load of its choices
    // is not waited for here
    L += gridDim.x;
    const bool more = find_place4<TM, TN>(p, ends, deal, L, false, next);
    const int choice = more ? choice4(p, next, tid) : -1;
    barrier();
    if (nk > 0) {
      o = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) a_part(i, h);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) b_part(i, h);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        qa[i] = scale_a(0, i);
        qb[i] = scale_b(0, i);
      }
      settle();  // the zeros, before an MFMA adds to them
      asm volatile("s_nop 15");
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      constexpr std::integral_constant<int, 0> zero{};
      constexpr std::integral_constant<int, 1> one{};
      constexpr std::integral_constant<int, 2> two{};
      int ks = 0;
      if constexpr (kGroup == 2) {  // two steps to a group, whose words stay for both
        for (; ks + 3 < nk; ks += 2) {
          step(ks, nk, yes, zero, zero);
          step(ks + 1, nk, yes, one, one);
        }
      }
      for (; ks < nk - 2; ++ks) step(ks, nk, yes, two, zero);
      for (; ks < nk; ++ks) step(ks, nk, no, two, zero);
      asm volatile("s_nop 15\n\ts_nop 15");  // the last MFMAs, before their results are read
      settle();
    }
    // the last step's barrier is past the last reads of both stages that count
    const Place4 done = cur;
    const int done_buf = buf;
    cur = next;
    nk = more && !cur.none ? all : 0;
    if (more) {
      buf ^= 1;
      src[buf][tid] = source4(p, choice);
      barrier();
      begin(cur, buf);
      preload(nk);
    }
    stored = row_in(done.m0, TM - 1, done.m_end) && done.n0 + TN <= p.N;
    if (stored) {
      output(done, done_buf, std::true_type{});
      if (more) arrive(nk, kStores);
    } else {
      output(done, done_buf, std::false_type{});
      if (more) arrive(nk, 0);
    }
    if (!more) return;
    clear();
  }
}

template <typename F>
bsq_status with_code(Code4 a, F&& f) {
  switch (a) {
    case Code4::e4m3: return f(std::integral_constant<int, 0>{});
    case Code4::e5m2: return f(std::integral_constant<int, 1>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

// Launches a product, with the events that the caller asked for, if any.
template <typename Kernel>
void launch_timed(Kernel k, dim3 grid, dim3 block, hipStream_t st, const Mx4Args& a) {
  const GemmEvents ev = take_gemm_events();
  if (ev.start != nullptr || ev.stop != nullptr) hipExtLaunchKernelGGL(k, grid, block, 0, st, ev.start, ev.stop, 0, a);
  else hipLaunchKernelGGL(k, grid, block, 0, st, a);
}

// Tile rows of all segments at most, or of the batch.
int64_t tile_rows(const Mx4Launch& L, int tm) { return L.offsets ? L.cap / tm + L.E + 1 : up_to(L.T, tm) * L.E; }

template <int MB, int NB, int W, int U>
bsq_status launch_few(const Mx4Launch& L, Mx4Args a, hipStream_t st) {
  return in_parts(tile_rows(L, 16 * MB) * up_to(L.N, 16 * NB), kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = int(first);
    return with_code(L.a, [&](auto fa) {
      launch_timed(k_mx4_few<decltype(fa)::value, MB, NB, W, U>, dim3(unsigned(n)), dim3(64 * W), st, a);
      return launch_status("mx4 product (few rows)");
    });
  });
}

template <int WM, int WN, int MB, int NB, int S, int KG, int U>
bsq_status launch_tile(const Mx4Launch& L, Mx4Args a, hipStream_t st) {
  return in_parts(tile_rows(L, 16 * MB * WM) * up_to(L.N, 16 * NB * WN), kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = int(first);
    return with_code(L.a, [&](auto fa) {
      constexpr int FA = decltype(fa)::value;
      const dim3 g = dim3(unsigned(n)), b = dim3(64 * WM * WN * KG);
      if (L.K % 128 == 0) launch_timed(k_mx4_tile<FA, WM, WN, MB, NB, S, KG, U, 1>, g, b, st, a);
      else launch_timed(k_mx4_tile<FA, WM, WN, MB, NB, S, KG, U, 0>, g, b, st, a);
      return launch_status("mx4 product");
    });
  });
}

bsq_status launch_big(const Mx4Launch& L, Mx4Args a, hipStream_t st) {
  // one workgroup to a CU, each going through its share of the tiles
  const int64_t grid = tile_rows(L, 256) * up_to(L.N, 256);
  const dim3 g = dim3(unsigned(grid < kCUs ? grid : kCUs)), b = dim3(256);
  return with_code(L.a, [&](auto fa) {
    constexpr int FA = decltype(fa)::value;
    if (L.out_bf16) launch_timed(k_mx4_big<FA, 1>, g, b, st, a);
    else launch_timed(k_mx4_big<FA, 0>, g, b, st, a);
    return launch_status("mx4 product (big tiles)");
  });
}

}  // namespace

bsq_status launch_mx4_product(const Mx4Launch& L, hipStream_t st) {
  const Mx4Args a{L.A, L.B, L.SA, L.SB, L.out, L.offsets, L.rows, L.T, L.cap, int(L.E), int(L.N), int(L.K), L.k,
                  L.out_bf16 ? 1 : 0, 0};
  const int64_t pitch_a = L.a == Code4::e2m1 ? L.K / 2 : L.K;
  switch (mx4_tile(Mx4Size{L.offsets != nullptr, L.rows != nullptr, L.T, L.cap, L.E, L.k, L.N, L.K})) {
    case Mx4Tile::few16x16: return L.K >= 128 * 8 * 4 ? launch_few<1, 1, 4, 8>(L, a, st) : launch_few<1, 1, 4, 4>(L, a, st);
    case Mx4Tile::few16x32: return L.K >= 128 * 8 * 4 ? launch_few<1, 2, 4, 8>(L, a, st) : launch_few<1, 2, 4, 4>(L, a, st);
    case Mx4Tile::few32x32: return launch_few<2, 2, 4, 4>(L, a, st);
    case Mx4Tile::t32x64: return launch_tile<1, 4, 2, 1, 3, 1, 1>(L, a, st);
    case Mx4Tile::t32x64g2: return launch_tile<1, 4, 2, 1, 2, 2, 2>(L, a, st);
    case Mx4Tile::t64x64g2: return launch_tile<2, 2, 2, 2, 3, 2, 1>(L, a, st);
    case Mx4Tile::t64x128g2: return launch_tile<2, 2, 2, 4, 3, 2, 1>(L, a, st);
    case Mx4Tile::t64x128: return launch_tile<2, 2, 2, 4, 2, 1, 1>(L, a, st);
    case Mx4Tile::t128x128: return launch_tile<4, 2, 2, 4, 2, 1, 1>(L, a, st);
    default:
      // gathered rows are addressed with 32 bits, and scales read 16 at a time
      // (experts' rows may be many more than the tokens; no contraction has none)
      if ((L.rows != nullptr && L.T * pitch_a >= (int64_t(1) << 32)) || L.T * (L.K / 32) < 16)
        return launch_tile<4, 2, 2, 4, 2, 1, 1>(L, a, st);
      return launch_big(L, a, st);
  }
}

}  // namespace bsq
