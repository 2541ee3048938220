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
#include "tiles.h"

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
// expert (or product) e.  `last`: no such expert, rows past the last segment.
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

// The workgroup's tile `L` in the order of tiles `rows_first`: along the
// columns first (few rows) or by tile_order.
template <int TM, int TN>
__device__ __forceinline__ bool find_place4(const Mx4Args& p, int lane, int L, bool along, Place4& t) {
  const int tiles_n = (p.N + TN - 1) / TN;
  int tm, tn, total;
  uint32_t before = 0, mine = 0;
  const int per = int((p.T + TM - 1) / TM);
  if (p.offsets != nullptr) total = tiles_total(Segments<TM>{p.offsets, p.E, p.cap}, lane, before, mine);
  else total = per * p.E;
  if (unsigned(L) >= unsigned(total) * unsigned(tiles_n)) return false;
  if (along) {
    tm = L / tiles_n;
    tn = L - tm * tiles_n;
  } else {
    tile_order(L, total, tiles_n, tm, tn);
  }
  if (p.offsets != nullptr) {
    const Segment s = find_tile(Segments<TM>{p.offsets, p.E, p.cap}, tm, before, mine);
    t.none = s.e >= p.E || p.T == 0;
    t.e = s.e < p.E ? s.e : 0;
    t.m0 = s.row0;
    t.m_end = s.end;
  } else {
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

// The row of A of a tile's row r, -1 for none.
__device__ __forceinline__ int source4(const Mx4Args& p, const Place4& t, int r) {
  if (!row_in(t.m0, r, t.m_end) || t.none) return -1;
  int f = t.m0 + r;
  if (p.rows != nullptr) {
    f = p.rows[f];
    if (f >= 0) f /= p.k;
  }
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
// joined through LDS in the waves' order.
template <int FA, int MB, int NB, int W>
__global__ void __launch_bounds__(64 * W) k_mx4_few(Mx4Args p) {
  constexpr int TM = 16 * MB, TN = 16 * NB, U = 4;
  constexpr int kPitch = TN + 4;  // of a row of sums, padded
  __shared__ __attribute__((aligned(16))) float red[W][TM][kPitch];
  __shared__ int src[TM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = scalar(tid >> 6);
  const View4<FA> view{p};
  Place4 t;
  if (!find_place4<TM, TN>(p, lane, p.first + int(blockIdx.x), true, t)) return;
  const int g = lane >> 4, r16 = lane & 15;
  const int nb = t.none ? 0 : p.K / 32;
  const uint8_t *pa[MB], *psa[MB], *pb[NB], *psb[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int s = source4(p, t, 16 * i + r16), row = s < 0 ? 0 : s;
    if (w == 0 && g == 0) src[16 * i + r16] = s;
    pa[i] = view.a(t.e) + row * view.pitch_a();
    psa[i] = view.sa(t.e) + row * view.pitch_s();
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t row = min(t.n0 + 16 * j + r16, p.N - 1);
    pb[j] = view.b(t.e) + row * view.pitch_b();
    psb[j] = view.sb(t.e) + row * view.pitch_s();
  }
  v4f acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int c0 = w * U; 4 * c0 < nb; c0 += W * U) {
    uint4 b[U][NB], a[U][MB][FA == 4 ? 1 : 2];
    int sb[U][NB], sa[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // block of the lane's scale, and of its chunks; past the end the last one
      const int at = 4 * (c0 + u) + g, k0 = min(at, nb - 1);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        b[u][j] = *reinterpret_cast<const uint4*>(pb[j] + 16 * k0);
        sb[u][j] = psb[j][k0];
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        sa[u][i] = psa[i][k0];
        if constexpr (FA == 4) {
          a[u][i][0] = *reinterpret_cast<const uint4*>(pa[i] + 16 * k0);
        } else {
          // 8 bits: 16 elements of block g / 2 and 16 of block 2 + g / 2
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 8 * (c0 + u) + 4 * h + g;  // chunk of 16 elements
            a[u][i][h] = *reinterpret_cast<const uint4*>(pa[i] + 16 * min(c, 2 * nb - 1));
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = 4 * (c0 + u) + g;
      if (4 * (c0 + u) + 4 > nb) {  // an end inside the chunk, or before it
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if (at >= nb) sa[u][i] = 127;
          if constexpr (FA == 4) {
            if (at >= nb) a[u][i][0] = zero;
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (8 * (c0 + u) + 4 * h + g >= 2 * nb) a[u][i][h] = zero;
          }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if (at >= nb) sb[u][j] = 127;
      }
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if constexpr (FA == 4) acc[j][i] = mfma4<FA>(wide(b[u][j]), wide(a[u][i][0]), acc[j][i], sb[u][j], sa[u][i]);
          else acc[j][i] = mfma4<FA>(wide(b[u][j]), wide(a[u][i][0], a[u][i][1]), acc[j][i], sb[u][j], sa[u][i]);
        }
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
// bytes (beside 8-bit A) lie two to a line.  Scales come as whole words: where
// K is no multiple of 128 a row's bytes start inside one, and one word more is
// read (AL 0).  A step waits for its own loads only.
template <int FA, int WM, int WN, int MB, int NB, int S, int AL>
__global__ void __launch_bounds__(64 * WM * WN, 1) k_mx4_tile(Mx4Args p) {
  constexpr int NW = WM * WN, TM = 16 * MB * WM, TN = 16 * NB * WN;
  constexpr int kStep = FA == 4 ? 256 : 128, kHalves = kStep / 128;
  constexpr int BA = 128, BB = kStep / 2;  // bytes of a row of a step
  constexpr int RB = 1024 / BB;            // rows of B of a load
  constexpr int LA = TM / 8 / NW, LB = TN / RB / NW;
  static_assert(TM % (8 * NW) == 0 && TN % (RB * NW) == 0 && NW % 2 == 0, "whole loads of every wave");
  constexpr int SM = (TM + 63) / 64 * 64, SR = SM + TN;  // rows of scales
  static_assert(TN % 64 == 0, "scale rows by the 64");
  constexpr int D = kHalves + (AL ? 0 : 1);       // words of a row's scales
  constexpr int LS = (SR / 64 * D + NW - 1) / NW;  // loads of them per wave
  constexpr int kStage = TM * BA + TN * BB;
  constexpr int kRowB = NB * 64 + 16;  // bytes of a staged output row of a wave, padded
  constexpr int kOut = NW * 16 * kRowB;
  constexpr int kAB = S * kStage > kOut ? S * kStage : kOut;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kAB];
  __shared__ __attribute__((aligned(16))) uint32_t lds_s[S][D][SR];
  __shared__ int src[TM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = scalar(tid >> 6);
  const View4<FA> view{p};
  Place4 t;
  if (!find_place4<TM, TN>(p, lane, p.first + int(blockIdx.x), false, t)) return;
  for (int r = tid; r < TM; r += 64 * NW) src[r] = source4(p, t, r);
  __syncthreads();
  const int nk = t.none ? 0 : (p.K + kStep - 1) / kStep;

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
  // whether the last step has not got the lane's chunk
  const int64_t last = int64_t(nk - 1) * BA, last_b = int64_t(nk - 1) * BB;
  const bool past_a = last + ca >= view.pitch_a(), past_b = last_b + cb >= view.pitch_b();
  const bool part = p.K % kStep != 0;
  // scales: 64 rows of one word to a load
  const int64_t sp = view.pitch_s();
  const uint64_t sa0 = reinterpret_cast<uint64_t>(view.sa(t.e));
  const int bm = int(sa0 & 3);  // a batch's scales need not start a word
  const i32x4 rsa = rsrc(reinterpret_cast<const uint8_t*>(sa0 - bm), (bm + p.T * sp + 3) & ~int64_t(3));
  const i32x4 rsb = rsrc(view.sb(t.e), p.N * sp);
  auto a_row = [&](int r) { return max(src[r], 0); };
  auto b_row = [&](int r) { return min(t.n0 + r, p.N - 1); };
  uint32_t so[LS], ls[LS];
  bool sA[LS];
#pragma unroll
  for (int q = 0; q < LS; ++q) {
    const int item = (w + NW * q) % (SR / 64 * D), grp = item / D, d = item % D;
    const int r = 64 * grp + lane;
    sA[q] = 64 * grp < SM;
    const uint32_t byte = sA[q] ? uint32_t(bm + a_row(min(r, TM - 1)) * sp) : uint32_t(b_row(r - SM) * sp);
    so[q] = (byte & ~3u) + 4u * uint32_t(d);
    ls[q] = lds_of(reinterpret_cast<const uint8_t*>(&lds_s[0][d][64 * grp]));
  }
  constexpr int kLoads = LA + LB + LS;
  const uint8_t* const zeros = kZeros;
  auto load = [&](int ks, int st) {
    const uint32_t at = uint32_t(st * kStage);
    if (part && ks == nk - 1) {
#pragma unroll
      for (int s = 0; s < LA; ++s) dma16(past_a ? zeros : pa[s] + last, la + at + uint32_t(1024 * NW * s));
#pragma unroll
      for (int s = 0; s < LB; ++s) dma16(past_b ? zeros : pb[s] + last_b, lb + at + uint32_t(1024 * NW * s));
    } else {
#pragma unroll
      for (int s = 0; s < LA; ++s) dma16(pa[s] + int64_t(ks) * BA, la + at + uint32_t(1024 * NW * s));
#pragma unroll
      for (int s = 0; s < LB; ++s) dma16(pb[s] + int64_t(ks) * BB, lb + at + uint32_t(1024 * NW * s));
    }
#pragma unroll
    for (int q = 0; q < LS; ++q)
      dma4(sA[q] ? rsa : rsb, so[q] + uint32_t(kStep / 32) * uint32_t(ks), ls[q] + uint32_t(st * D * SR * 4));
  };

  const int wm = w % WM, wn = w / WM, g = lane >> 4, r16 = lane & 15;
  const int x8 = r16 >> 1;  // what a row's chunks are XORed with
  // where a lane's scale bytes start inside the first word of its rows
  int ma[MB], mb = 0;
#pragma unroll
  for (int i = 0; i < MB; ++i) ma[i] = AL ? 0 : int((unsigned(bm) + unsigned(a_row(16 * MB * wm + 16 * i + r16)) * unsigned(sp)) & 3u);
  if (!AL) mb = int((unsigned(b_row(16 * NB * wn + r16)) * unsigned(sp)) & 3u);
  v4f acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int ks = 0; ks < min(nk, S - 1); ++ks) load(ks, ks);

  int st = 0;
  for (int ks = 0; ks < nk; ++ks) {
    // S - 2 steps stay under way; near the end, where fewer are, all are waited for
    if (ks + S - 2 < nk) __builtin_amdgcn_s_waitcnt(vmcnt((S - 2) * kLoads));
    else __builtin_amdgcn_s_waitcnt(vmcnt(0));
    barrier();
    // past the barrier nobody reads the stage before this one
    if (ks + S - 1 < nk) load(ks + S - 1, st == 0 ? S - 1 : st - 1);
    const uint8_t* ta = lds + st * kStage;
    const uint8_t* tb = ta + TM * BA;
    const uint32_t(*ss)[SR] = lds_s[st];
    auto scale = [&](int row, int mis, int block) -> int {  // byte `block` of a row's scales of the step
      if (AL) return int((ss[block >> 2][row] >> (8 * (block & 3))) & 0xFFu);
      const int byte = mis + block;
      return reinterpret_cast<const uint8_t*>(&ss[byte >> 2][row])[byte & 3];
    };
    int qa[kHalves][MB], qb[kHalves][NB];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
#pragma unroll
      for (int i = 0; i < MB; ++i) qa[h][i] = scale(16 * MB * wm + 16 * i + r16, ma[i], 4 * h + g);
#pragma unroll
      for (int j = 0; j < NB; ++j) qb[h][j] = scale(SM + 16 * NB * wn + 16 * j + r16, mb, 4 * h + g);
    }
    if (part && ks == nk - 1) {
      const int left = p.K / 32 - ks * (kStep / 32);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const bool past = 4 * h + g >= left;
#pragma unroll
        for (int i = 0; i < MB; ++i) qa[h][i] = past ? 127 : qa[h][i];
#pragma unroll
        for (int j = 0; j < NB; ++j) qb[h][j] = past ? 127 : qb[h][j];
      }
    }
    auto chunk = [&](const uint8_t* tile, int row, int c) {  // of a 128-byte row
      return *reinterpret_cast<const uint4*>(tile + row * 128 + 16 * (c ^ x8));
    };
    auto bfrag = [&](int h, int j) {
      const int row = 16 * NB * wn + 16 * j + r16;
      if constexpr (BB == 128) return wide(chunk(tb, row, 4 * h + g));
      else return wide(*reinterpret_cast<const uint4*>(tb + (row >> 1) * 128 + 64 * (row & 1) + 16 * (g ^ ((row >> 2) & 3))));
    };
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      v8i fa[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int row = 16 * MB * wm + 16 * i + r16;
        if constexpr (FA == 4) fa[i] = wide(chunk(ta, row, 4 * h + g));
        else fa[i] = wide(chunk(ta, row, g), chunk(ta, row, 4 + g));
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const v8i fb = bfrag(h, j);
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = mfma4<FA>(fb, fa[i], acc[j][i], qb[h][j], qa[h][i]);
      }
    }
    st = st == S - 1 ? 0 : st + 1;
  }

  // ---- out: 16 rows of the wave at a time through LDS, so that a store
  // instruction writes whole rows of the wave's columns
  uint8_t* const stg = lds + w * 16 * kRowB;
  constexpr int LPR = 4 * NB, RPI = 64 / LPR;
  static_assert(64 % LPR == 0, "whole rows per instruction");
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NB; ++j) *reinterpret_cast<v4f*>(stg + r16 * kRowB + (16 * j + 4 * g) * 4) = acc[j][i];
    __syncthreads();
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

template <typename F>
bsq_status with_code(Code4 a, F&& f) {
  switch (a) {
    case Code4::e4m3: return f(std::integral_constant<int, 0>{});
    case Code4::e5m2: return f(std::integral_constant<int, 1>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

// Tile rows of all segments at most, or of the batch.
int64_t tile_rows(const Mx4Launch& L, int tm) { return L.offsets ? L.cap / tm + L.E + 1 : up_to(L.T, tm) * L.E; }

template <int MB, int NB, int W>
bsq_status launch_few(const Mx4Launch& L, Mx4Args a, hipStream_t st) {
  return in_parts(tile_rows(L, 16 * MB) * up_to(L.N, 16 * NB), kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = int(first);
    return with_code(L.a, [&](auto fa) {
      hipLaunchKernelGGL((k_mx4_few<decltype(fa)::value, MB, NB, W>), dim3(unsigned(n)), dim3(64 * W), 0, st, a);
      return launch_status("mx4 product (few rows)");
    });
  });
}

template <int WM, int WN, int MB, int NB, int S>
bsq_status launch_tile(const Mx4Launch& L, Mx4Args a, hipStream_t st) {
  return in_parts(tile_rows(L, 16 * MB * WM) * up_to(L.N, 16 * NB * WN), kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = int(first);
    return with_code(L.a, [&](auto fa) {
      constexpr int FA = decltype(fa)::value;
      const dim3 g = dim3(unsigned(n)), b = dim3(64 * WM * WN);
      if (L.K % 128 == 0) hipLaunchKernelGGL((k_mx4_tile<FA, WM, WN, MB, NB, S, 1>), g, b, 0, st, a);
      else hipLaunchKernelGGL((k_mx4_tile<FA, WM, WN, MB, NB, S, 0>), g, b, 0, st, a);
      return launch_status("mx4 product");
    });
  });
}

}  // namespace

bsq_status launch_mx4_product(const Mx4Launch& L, hipStream_t st) {
  const Mx4Args a{L.A, L.B, L.SA, L.SB, L.out, L.offsets, L.rows, L.T, L.cap, int(L.E), int(L.N), int(L.K), L.k,
                  L.out_bf16 ? 1 : 0, 0};
  const int64_t rows = L.offsets ? (L.rows && L.T < L.cap / L.k ? L.T * L.k : L.cap) / L.E : L.T;
  if (rows <= 16 && L.cap <= (1 << 20)) return launch_few<1, 2, 8>(L, a, st);
  return launch_tile<2, 2, 2, 4, 2>(L, a, st);
}

}  // namespace bsq
