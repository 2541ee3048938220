// The experts' products over ragged rows, block-scaled in 8 bits (E8M0
// scales per 32 elements), one launch for all experts.
//
//   product  out[r, n] = sum_k A[src(r), k] B[e, n, k] for the rows r of
//            expert e's segment [offsets[e], offsets[e + 1]), where
//            src(r) = rows[r] / topk (or r): the gather of the tokens is
//            the product's own load.  Rows without a choice and rows past
//            the last segment are written as zeros.
//   wgrad    dW[e, n, k] = sum over r of expert e's segment of
//            dyt[n, r] xt[k, r].
//
// The segments are known on the device only.  A workgroup finds its tile by
// a scan of the offsets; the grid covers the most tiles that any split of
// `cap` rows over E experts can have, and what is left over ends at once.
// Offsets and row numbers are clamped to their arrays, so that no content of
// theirs makes an access out of range.
//
// One tile: WM x WN waves, each with MB x NB blocks of 16 x 16
// (v_mfma_scale_f32_16x16x128_f8f6f4, both E8M0 scales applied in the matrix
// core, float32 accumulators).  K goes in steps of 128 bytes through two LDS
// stages filled by direct loads, 16-byte chunks XOR-swizzled over the rows so
// that a fragment read spreads over the banks; the next step's loads are
// issued between this step's MFMAs.  The scales of four steps come as one
// 16-byte piece per row.  The MFMA's first operand is the B fragment, so that
// a lane's four results are four neighbours of one output row.
#include "moe.h"

namespace bsq {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int BK = 128;

struct MoeArgs {
  const uint8_t *A, *B, *SA, *SB;
  void* out;
  const int32_t *offsets, *rows;
  int64_t T, cap;
  int E, N, K, k;
};

// Buffer resource of `records` bytes (in range 0 .. 2^32 - 1) from `base`;
// reads past it give zeros.
__device__ __forceinline__ i32x4 rsrc(const uint8_t* base, int64_t records) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t n = uint32_t(records < 0 ? 0 : (records > int64_t(0xFFFFFFFF) ? int64_t(0xFFFFFFFF) : records));
  return i32x4{__builtin_amdgcn_readfirstlane(int(uint32_t(b))),
               __builtin_amdgcn_readfirstlane(int(uint32_t(b >> 32) & 0xFFFFu)),
               __builtin_amdgcn_readfirstlane(int(n)), 0x00020000};
}

// 16 bytes per lane straight into LDS: lane i fills [lds + 16 i, + 16).  In
// inline asm, so that the compiler does not order it against the reads of
// the other stage; the caller waits with vmcnt before the barrier that
// publishes the stage.  No register is written.
__device__ __forceinline__ void dma16(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void dma16(i32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r)
               : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_of(const uint8_t* p) {
  return __builtin_amdgcn_readfirstlane(
      uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)(p))));
}

__device__ __forceinline__ v8i frag(const uint8_t* tile, int off0, int off1) {
  const uint4 lo = *reinterpret_cast<const uint4*>(tile + off0);
  const uint4 hi = *reinterpret_cast<const uint4*>(tile + off1);
  return v8i{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
}

__device__ __forceinline__ int bounded(int v, int64_t cap) { return v < 0 ? 0 : (v > cap ? int(cap) : v); }

// Segment of the mt-th tile of TM rows when every segment is cut into tiles
// from its first row: expert (E: the rows past the last segment), first row
// and end.  `total` is the number of tiles.  Every wave computes it alone:
// lane l sums the tiles of segments [l c, (l + 1) c), a scan over the lanes
// finds the lane, and that lane's segments are walked.
struct Segment {
  int e, row0, end;
};
__device__ __forceinline__ int tiles_total(const MoeArgs& a, int tm, int lane, int& mine_before, int& mine) {
  const int S = a.E + 1, c = (S + 63) / 64;
  int n = 0;
  for (int i = lane * c; i < min((lane + 1) * c, S); ++i) {
    const int lo = bounded(a.offsets[i], a.cap), hi = i < a.E ? bounded(a.offsets[i + 1], a.cap) : int(a.cap);
    n += hi > lo ? (hi - lo + tm - 1) / tm : 0;
  }
  int s = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  mine_before = s - n;
  mine = n;
  return __builtin_amdgcn_readlane(s, 63);
}
__device__ __forceinline__ Segment find_tile(const MoeArgs& a, int tm, int lane, int mt, int mine_before, int mine) {
  const int S = a.E + 1, c = (S + 63) / 64;
  const uint64_t here = __ballot(mt >= mine_before && mt < mine_before + mine);
  const int l = here ? __ffsll((unsigned long long)here) - 1 : 63;
  int left = mt - __builtin_amdgcn_readlane(mine_before, l);
  Segment s{a.E, int(a.cap), int(a.cap)};
  for (int i = l * c; i < min((l + 1) * c, S); ++i) {
    const int lo = bounded(a.offsets[i], a.cap), hi = i < a.E ? bounded(a.offsets[i + 1], a.cap) : int(a.cap);
    const int n = hi > lo ? (hi - lo + tm - 1) / tm : 0;
    if (left < n) {
      s = Segment{i, lo + left * tm, hi};
      break;
    }
    left -= n;
  }
  s.e = __builtin_amdgcn_readfirstlane(s.e);
  s.row0 = __builtin_amdgcn_readfirstlane(s.row0);
  s.end = __builtin_amdgcn_readfirstlane(s.end);
  return s;
}

// Tile order: workgroups are dealt to the 8 XCDs round-robin by linear id,
// and each XCD has its own L2, so XCD x takes the x-th contiguous eighth of
// an order that walks bands of kBand tile rows column by column.
__device__ __forceinline__ void tile_order(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kBand = 4;
  const int T = tiles_m * tiles_n, per = T / 8;
  const int t = L < 8 * per ? (L % 8) * per + L / 8 : L;
  const int band = t / (kBand * tiles_n);
  const int rows = min(kBand, tiles_m - band * kBand);
  const int in = t - band * kBand * tiles_n;
  tm = band * kBand + in % rows;
  tn = in / rows;
}

// A tile's operands: rows of A (a row number per tile row, clamped) and B.
template <int WM, int WN, int MB, int NB, int FA, int OUT_BF16, int WGRAD>
__global__ void __launch_bounds__(64 * WM * WN, 1) k_moe_gemm(MoeArgs p) {
  constexpr int NW = WM * WN;
  constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN;
  constexpr int SA_ = TM / 8 / NW, SB_ = TN / 8 / NW;  // 8-row slices per wave
  static_assert(TM % (8 * NW) == 0 && TN % (8 * NW) == 0, "whole slices");
  static_assert(TM % 64 == 0 && TN % 64 == 0, "scale rows by the 64");
  constexpr int kStage = (TM + TN) * BK;
  constexpr int kRowB = NB * 64 + 16;  // bytes of a staged output row of a wave, padded
  constexpr int kOut = NW * 16 * kRowB;
  constexpr int kAB = 2 * kStage > kOut ? 2 * kStage : kOut;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kAB];
  __shared__ __attribute__((aligned(16))) uint32_t lds_s[2][(TM + TN) * 4];
  __shared__ int src[TM];  // row of A of each tile row, -1: none

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = p.N;
  int m0, m_end, n0, M_total;   // output rows [m0, m_end) and first column
  int64_t pitch;                // bytes per row of A and B along the contraction
  int64_t k0 = 0;               // first byte of the contraction
  int nk;
  int64_t out0;                 // first element of the output matrix
  const uint8_t *A = p.A, *B = p.B, *SA = p.SA, *SB = p.SB;
  int N_total = N;
  if (WGRAD) {
    const int tiles_m = (N + TM - 1) / TM, tiles_n = (p.K + TN - 1) / TN;
    const int per = tiles_m * tiles_n, all = per * p.E;
    int L = blockIdx.x;
    const int eighth = all / 8;
    if (L < 8 * eighth) L = (L % 8) * eighth + L / 8;
    const int e = L / per, in = L - e * per;
    m0 = in / tiles_n * TM;
    n0 = in % tiles_n * TN;
    m_end = M_total = N;
    N_total = p.K;
    pitch = p.cap;
    const int lo = bounded(p.offsets[e], p.cap) / BK, hi = bounded(p.offsets[e + 1], p.cap) / BK;
    k0 = int64_t(lo) * BK;
    nk = max(hi - lo, 0);
    out0 = int64_t(e) * N * p.K;
  } else {
    int before, mine;
    const int tiles_m = tiles_total(p, TM, lane, before, mine), tiles_n = (N + TN - 1) / TN;
    if (blockIdx.x >= unsigned(tiles_m) * unsigned(tiles_n)) return;
    int tm, tn;
    tile_order(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const Segment s = find_tile(p, TM, lane, tm, before, mine);
    m0 = s.row0;
    m_end = s.end;
    n0 = tn * TN;
    M_total = int(p.T);
    pitch = p.K;
    nk = s.e < p.E && p.T > 0 ? p.K / BK : 0;
    B += int64_t(s.e < p.E ? s.e : 0) * N * p.K;
    SB += int64_t(s.e < p.E ? s.e : 0) * N * (p.K / 32);
    out0 = 0;
    for (int r = tid; r < TM; r += 64 * NW) {
      int t = -1;
      if (m0 + r < m_end && nk > 0) {
        t = p.rows != nullptr ? p.rows[m0 + r] : m0 + r;
        if (p.rows != nullptr && t >= 0) t /= p.k;
        if (t >= M_total) t = -1;
      }
      src[r] = t;
    }
    __syncthreads();
  }
  auto a_row = [&](int r) {  // row of A of tile row r, always inside A
    if (WGRAD) return min(m0 + r, M_total - 1);
    return max(src[r], 0);
  };

  // ---- loads: lane i of an 8-row slice fills row i / 8, chunk i % 8 of it
  // with the chunk that the swizzle keeps there
  const int lrow = lane >> 3, chunk = 16 * ((lane & 7) ^ lrow);
  const uint8_t *pa[SA_], *pb[SB_];
#pragma unroll
  for (int s = 0; s < SA_; ++s) pa[s] = A + int64_t(a_row(8 * (w + NW * s) + lrow)) * pitch + k0 + chunk;
#pragma unroll
  for (int s = 0; s < SB_; ++s)
    pb[s] = B + int64_t(min(n0 + 8 * (w + NW * s) + lrow, N_total - 1)) * pitch + k0 + chunk;
  const uint32_t la = lds_of(lds + 8 * w * BK), lb = lds_of(lds + TM * BK + 8 * w * BK);
  // step ks (past the last one: the last again, into a stage nobody reads)
  auto load_a = [&](int ks, int st, int s) {
    dma16(pa[s] + int64_t(min(ks, nk - 1)) * BK, la + uint32_t(st * kStage + 8 * NW * s * BK));
  };
  auto load_b = [&](int ks, int st, int s) {
    dma16(pb[s] + int64_t(min(ks, nk - 1)) * BK, lb + uint32_t(st * kStage + 8 * NW * s * BK));
  };

  // ---- scales: rows 64 s .. of A, then of B, four steps (16 bytes) each
  const int64_t spitch = pitch / 32;
  constexpr int SS = (TM + TN) / 64, SPW = (SS + NW - 1) / NW;
  uint32_t soff[SPW];
  const int64_t n_sa = (WGRAD ? int64_t(N) : p.T) * spitch, n_sb = int64_t(N_total) * spitch;
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
    const int s = w + NW * i, r = 64 * s + lane;
    const int64_t row = r < TM ? a_row(min(r, TM - 1)) : min(n0 + r - TM, N_total - 1);
    soff[i] = uint32_t(row * spitch + k0 / 32);
  }
  const uint32_t ls = lds_of(reinterpret_cast<const uint8_t*>(&lds_s[0][0]));
  auto load_scales = [&](int q) {
#pragma unroll
    for (int i = 0; i < SPW; ++i) {
      const int s = w + NW * i;
      if (s < SS)
        dma16(s < TM / 64 ? rsrc(SA, n_sa) : rsrc(SB, n_sb), soff[i] + 16u * uint32_t(q),
              ls + uint32_t((q & 1) * (TM + TN) * 16 + 64 * s * 16));
    }
  };

  const int wm = w % WM, wn = w / WM, g = lane >> 4, r16 = lane & 15;
  const int c0 = 16 * (g ^ (r16 & 7)), c1 = 16 * ((g + 4) ^ (r16 & 7));
  v4f acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};

  if (nk > 0) {
#pragma unroll
    for (int s = 0; s < SA_; ++s) load_a(0, 0, s);
#pragma unroll
    for (int s = 0; s < SB_; ++s) load_b(0, 0, s);
    load_scales(0);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();

  for (int ks = 0; ks < nk; ++ks) {
    const int st = ks & 1;
    if ((ks & 3) == 3 && ks + 1 < nk) load_scales((ks + 1) >> 2);
    const uint8_t* ta = lds + st * kStage;
    const uint8_t* tb = ta + TM * BK;
    const uint32_t* ss = &lds_s[(ks >> 2) & 1][ks & 3];
    uint32_t qa[MB], qb[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) qa[i] = ss[(16 * MB * wm + 16 * i + r16) * 4];
#pragma unroll
    for (int j = 0; j < NB; ++j) qb[j] = ss[(TM + 16 * NB * wn + 16 * j + r16) * 4];
    __builtin_amdgcn_sched_barrier(0);
    auto bfrag = [&](int j) {
      const int row = 16 * NB * wn + 16 * j + r16;
      return frag(tb, row * BK + c0, row * BK + c1);
    };
    v8i fb[2] = {bfrag(0), {}};
    v8i fa[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row = 16 * MB * wm + 16 * i + r16;
      fa[i] = frag(ta, row * BK + c0, row * BK + c1);
    }
    if (NB > 1) fb[1] = bfrag(1);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      // two slices of the next step at the head of each block of columns
#pragma unroll
      for (int s = 0; s < SA_; ++s)
        if (s / ((SA_ + NB - 1) / NB) == j) load_a(ks + 1, st ^ 1, s);
#pragma unroll
      for (int s = 0; s < SB_; ++s)
        if (s / ((SB_ + NB - 1) / NB) == j) load_b(ks + 1, st ^ 1, s);
      v8i next{};
      if (j + 2 < NB) next = bfrag(j + 2);
      const int b = int((qb[j] >> (8 * g)) & 0xFFu);
#pragma unroll
      for (int i = 0; i < MB; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[0], fa[i], acc[j][i], 0, FA, 0, b, 0,
                                                                      int((qa[i] >> (8 * g)) & 0xFFu));
      fb[0] = fb[1];
      fb[1] = next;
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
  }

  // ---- out: 16 rows of the wave at a time through LDS, so that a store
  // instruction writes whole rows of the wave's columns
  uint8_t* const stg = lds + w * 16 * kRowB;
  constexpr int LPR = 4 * NB;          // lanes per row, four columns each
  constexpr int RPI = 64 / LPR > 0 ? 64 / LPR : 1;
  static_assert(64 % LPR == 0, "whole rows per instruction");
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<v4f*>(stg + r16 * kRowB + (16 * j + 4 * g) * 4) = acc[j][i];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 16 / RPI; ++t) {
      const int rr = RPI * t + lane / LPR, cc = 4 * (lane % LPR);
      const int tr = 16 * MB * wm + 16 * i + rr;
      const int m = m0 + tr, n = n0 + 16 * NB * wn + cc;
      v4f v = *reinterpret_cast<const v4f*>(stg + rr * kRowB + cc * 4);
      if (!WGRAD && src[tr] < 0) v = v4f{0.f, 0.f, 0.f, 0.f};
      if (m < m_end && n < N_total) {
        const int64_t o = out0 + int64_t(m) * N_total + n;
        if (OUT_BF16) {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          const uint32_t lo = encode_bf16(v[0]) | (encode_bf16(v[1]) << 16);
          const uint32_t hi = encode_bf16(v[2]) | (encode_bf16(v[3]) << 16);
          __builtin_nontemporal_store(u32x2{lo, hi}, reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + o));
        } else {
          __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(static_cast<float*>(p.out) + o));
        }
      }
    }
  }
}

template <int WM, int WN, int MB, int NB, int WGRAD>
bsq_status launch(const MoeArgs& a, bool e5m2, bool bf16, int64_t grid, hipStream_t st) {
  const dim3 g = dim3(unsigned(grid)), b = dim3(64 * WM * WN);
  switch ((e5m2 ? 1 : 0) | (bf16 ? 2 : 0)) {
    case 0: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, 0, 0, WGRAD>), g, b, 0, st, a); break;
    case 1: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, 1, 0, WGRAD>), g, b, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, 0, 1, WGRAD>), g, b, 0, st, a); break;
    default: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, 1, 1, WGRAD>), g, b, 0, st, a);
  }
  return launch_status(WGRAD ? "moe_wgrad" : "moe_matmul");
}

MoeArgs args_of(const MoeGemmLaunch& L) {
  return MoeArgs{L.A, L.B, L.SA, L.SB, L.out, L.offsets, L.rows, L.T, L.cap, L.E, int(L.N), int(L.K), L.k};
}

int64_t up_to(int64_t v, int64_t m) { return (v + m - 1) / m; }

}  // namespace

bsq_status launch_moe_product(const MoeGemmLaunch& L, hipStream_t st) {
  const MoeArgs a = args_of(L);
  // a segment's last tile may be part full: at most one such tile for each
  // expert and for the rows past the last segment
  auto grid = [&](int tm, int tn) { return (L.cap / tm + L.E + 1) * up_to(L.N, tn); };
  if (L.cap / L.E >= 512) return launch<4, 2, 4, 8, 0>(a, L.a_e5m2, L.out_bf16, grid(256, 256), st);
  if (L.cap / L.E >= 64) return launch<2, 2, 4, 4, 0>(a, L.a_e5m2, L.out_bf16, grid(128, 128), st);
  return launch<2, 2, 2, 2, 0>(a, L.a_e5m2, L.out_bf16, grid(64, 64), st);
}

bsq_status launch_moe_wgrad(const MoeGemmLaunch& L, hipStream_t st) {
  const MoeArgs a = args_of(L);
  const int64_t big = up_to(L.N, 256) * up_to(L.K, 256) * L.E;
  if (big >= 256) return launch<4, 2, 4, 8, 1>(a, L.a_e5m2, L.out_bf16, big, st);
  return launch<2, 2, 4, 4, 1>(a, L.a_e5m2, L.out_bf16, up_to(L.N, 128) * up_to(L.K, 128) * L.E, st);
}

}  // namespace bsq
