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
// a scan of the offsets; there are tiles for the most that any split of `cap`
// rows over E experts can have, and a workgroup without one ends at once.
// Offsets and row numbers are clamped to their arrays, so that no content of
// theirs makes an access out of range.
//
// Two kernels.  k_moe_big takes 256 x 256 tiles (many rows to an expert);
// k_moe_gemm takes the rest: WM x WN waves, each with MB x NB blocks of 16 x
// 16 (v_mfma_scale_f32_16x16x128_f8f6f4, both E8M0 scales applied in the
// matrix core, float32 accumulators).  K goes in steps of 128 bytes through a
// ring of S LDS stages filled by direct loads, 16-byte chunks XOR-swizzled
// over the rows so that a fragment read spreads over the banks.  A step waits
// for its own loads only (they retire in order), so that S - 2 more steps
// stay under way.  The MFMA's first operand is the B fragment, so that a
// lane's four results are four neighbours of one output row.
//
// Measured (MI355X): 65536 rows over 32 experts, N 4096, K 2048: 545 us, 2.02
// PFLOP/s; the weight gradients of 32768 rows over 16 experts, N = K = 2048:
// 148 us, 1.86 PFLOP/s; 65536 own rows in e5m2, N 2048, K 4096: 535 us.  A big
// tile's 16 steps take 47 k cycles, 2950 a step where its 256 MFMAs take 2048
// (with every load a hit in the L2 2700, without loads 2500); the rest of a
// tile 10.6 k: search 1.4, addresses 1.0, waits 0.4, output with the next
// tile's first loads 7.8.  The clock is at 1.8 GHz meanwhile (cycles over time);
// pure MFMAs on such operands run at 16 - 19 ns per 16 x 16 x 128, not the 13.3
// of 2.4 GHz.  8 tokens over 32 experts (N 4096, K 2048): 30 - 34 us, 5.1 - 5.8
// TB/s of weights.
#include "moe.h"
#include "moe_index.h"

#include <type_traits>

namespace bsq {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int BK = 128;

struct MoeArgs {
  const uint8_t *A, *B, *SA, *SB;
  void* out;
  const int32_t *offsets, *rows;
  int64_t T, cap;
  int E, N, K, k;
  int first;  // workgroup of this launch (k_moe_gemm)
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

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t scalar(int64_t v) {
  return int64_t(uint64_t(uint32_t(scalar(int(v)))) | (uint64_t(uint32_t(scalar(int(v >> 32)))) << 32));
}
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* v) {
  return reinterpret_cast<const uint8_t*>(scalar(reinterpret_cast<int64_t>(v)));
}

// 16 bytes per lane straight into LDS: lane i fills [lds + 16 i, + 16).  In
// inline asm, so that the compiler does not order it against the reads of
// the other stage; the caller waits with vmcnt before the barrier that
// publishes the stage.  No register is written.  The compiler does not know
// what these are, so the waits that the hardware leaves to software are in
// them: one state from m0 to its use, five from a descriptor that a vector
// instruction may have written.
__device__ __forceinline__ void dma16(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void dma16(i32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(scalar(int(lds))), "v"(voff), "s"(r)
               : "memory");
}
// 4 bytes per lane: lane i fills [lds + 4 i, + 4).
__device__ __forceinline__ void dma4(i32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(scalar(int(lds))), "v"(voff), "s"(r)
               : "memory");
}
// From a 32-bit offset to a base in scalar registers, to `at` (a constant
// where it is inlined) past lds.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds, int at) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base), "i"(at)
               : "memory", "scc");
}

// The same, to be dropped from the L2 first.
__device__ __forceinline__ void dma16_stream(const uint8_t* base, uint32_t off, uint32_t lds, int at) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
               :
               : "s"(lds), "v"(off), "s"(base), "i"(at)
               : "memory", "scc");
}

// s_waitcnt's operand: at most n vector memory operations under way.
constexpr int vmcnt(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }
// A barrier that no access of the compiler's moves across.
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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

// The tiles of all segments (`total`), and the segment of the mt-th.  Every
// wave computes it alone: lane l sums the tiles of its share of the segments,
// a scan over the lanes finds the lane, and that lane's segments are walked.
template <int TM>
__device__ __forceinline__ Segments<TM> segments(const MoeArgs& a) {
  return Segments<TM>{a.offsets, a.E, a.cap};
}
template <int TM>
__device__ __forceinline__ int tiles_total(const MoeArgs& a, int lane, uint32_t& mine_before, uint32_t& mine) {
  mine = segments<TM>(a).lane_tiles(lane);
  uint32_t s = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  mine_before = s - mine;
  const uint32_t total = uint32_t(__builtin_amdgcn_readlane(int(s), 63)), limit = uint32_t(segments<TM>(a).limit());
  return scalar(int(total < limit ? total : limit));
}
template <int TM>
__device__ __forceinline__ Segment find_tile(const MoeArgs& a, int mt, uint32_t mine_before, uint32_t mine) {
  const uint64_t here = __ballot(Segments<TM>::has(mine_before, mine, mt));
  const int l = here ? __ffsll((unsigned long long)here) - 1 : 63;
  Segment s = segments<TM>(a).at(l, mt - __builtin_amdgcn_readlane(int(mine_before), l));
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

// What a workgroup computes: output rows [m0, m_end) and columns from n0 of
// expert e, over nk steps of the contraction from byte k0 on.
struct Place {
  int e, m0, m_end, n0, nk, k0;
};
// The operands and the output that hold it.
template <int WGRAD>
struct View {
  const MoeArgs& p;
  __device__ __forceinline__ int rows_a() const { return WGRAD ? p.N : int(p.T); }
  __device__ __forceinline__ int rows_b() const { return WGRAD ? p.K : p.N; }  // and columns of out
  __device__ __forceinline__ int64_t pitch() const { return WGRAD ? p.cap : int64_t(p.K); }  // bytes per row of both
  __device__ __forceinline__ const uint8_t* b(const Place& t) const {
    return p.B + (WGRAD ? 0 : int64_t(t.e) * p.N * p.K);
  }
  __device__ __forceinline__ const uint8_t* sb(const Place& t) const {
    return p.SB + (WGRAD ? 0 : int64_t(t.e) * p.N * (p.K / 32));
  }
  __device__ __forceinline__ int64_t out0(const Place& t) const { return WGRAD ? int64_t(t.e) * p.N * p.K : 0; }
};

// What a lane knows of the tiles of all experts, for find_place.
//   product  tiles_total's numbers (`total`: all tiles)
//   wgrad    `total` 1: the experts' tiles go to the XCDs in chunks of 32, a
//            chunk's tiles to the XCD's 32 workgroups, the chunks in the order
//            of their contractions' lengths, back and forth over the XCDs, so
//            that each gets as many steps (expert e's rank is `before` of lane
//            e).  0: an eighth of the tiles to each XCD.
struct Deal {
  int total;
  uint32_t before, mine;
};
template <int TM, int TN, int WGRAD>
__device__ __forceinline__ Deal deal_tiles(const MoeArgs& p, int lane) {
  Deal d{0, 0, 0};
  if (!WGRAD) {
    d.total = tiles_total<TM>(p, lane, d.before, d.mine);
    return d;
  }
  // 16 experts of 2048 x 2048 over 32768 rows, segments of 0.5 to 2 times the
  // mean: 165 us against 213 by eighths (one XCD had 1.38 times the mean's steps)
  if (gridDim.x != kCUs || !dealt(((p.N + TM - 1) / TM) * ((p.K + TN - 1) / TN), p.E)) return d;
  d.total = 1;
  int len = -1;
  if (lane < p.E) len = max(bounded(p.offsets[lane + 1], p.cap) / BK - bounded(p.offsets[lane], p.cap) / BK, 0);
  for (int e = 0; e < p.E; ++e) {
    const int o = __builtin_amdgcn_readlane(len, e);
    d.before += o > len || (o == len && e < lane) ? 1 : 0;
  }
  return d;
}

// Where the workgroup's tile `L` is (L: blockIdx.x plus multiples of
// gridDim.x; moved on past tiles that are not there); false if there is none.
template <int TM, int TN, int WGRAD>
__device__ __forceinline__ bool find_place(const MoeArgs& p, int lane, const Deal& d, int& L, Place& t) {
  const int rows_b = View<WGRAD>{p}.rows_b(), tiles_n = (rows_b + TN - 1) / TN;
  if (WGRAD) {
    const int per = (p.N + TM - 1) / TM * tiles_n, all = per * p.E;
    int in;
    if (d.total) {
      const int chunks = (per + 31) / 32, x = L & 7;
      for (;; L += kCUs) {
        const int i = L / int(kCUs), q = 8 * i + ((i & 1) ? 7 - x : x);
        if (q >= chunks * p.E) return false;
        in = q % chunks * 32 + (L % int(kCUs)) / 8;
        if (in >= per) continue;
        t.e = __ffsll((unsigned long long)__ballot(lane < p.E && int(d.before) == q / chunks)) - 1;
        break;
      }
    } else {
      if (L >= all) return false;
      const int eighth = all / 8, T = L < 8 * eighth ? (L % 8) * eighth + L / 8 : L;
      t.e = T / per;
      in = T % per;
    }
    t.e = scalar(t.e);
    t.m0 = in / tiles_n * TM;
    t.n0 = in % tiles_n * TN;
    t.m_end = p.N;
    const int lo = bounded(p.offsets[t.e], p.cap) / BK, hi = bounded(p.offsets[t.e + 1], p.cap) / BK;
    t.k0 = lo * BK;
    t.nk = max(hi - lo, 0);
  } else {
    if (unsigned(L) >= unsigned(d.total) * unsigned(tiles_n)) return false;
    int tm, tn;
    tile_order(L, d.total, tiles_n, tm, tn);
    const Segment s = find_tile<TM>(p, tm, d.before, d.mine);
    t.e = s.e < p.E ? s.e : 0;
    t.m0 = s.row0;
    t.m_end = s.end;
    t.n0 = tn * TN;
    t.k0 = 0;
    t.nk = s.e < p.E && p.T > 0 ? p.K / BK : 0;
  }
  t.e = scalar(t.e);
  t.m0 = scalar(t.m0);
  t.m_end = scalar(t.m_end);
  t.n0 = scalar(t.n0);
  t.nk = scalar(t.nk);
  t.k0 = scalar(t.k0);
  return true;
}

// The row of A of a tile's row r, -1 for none (product only): the choice at
// the row, and the row of it.
__device__ __forceinline__ int choice_at(const MoeArgs& p, const Place& t, int r) {
  if (!row_in(t.m0, r, t.m_end) || t.nk == 0) return -1;
  return p.rows != nullptr ? p.rows[t.m0 + r] : t.m0 + r;
}
__device__ __forceinline__ int source_of(const MoeArgs& p, int choice) {
  const int f = p.rows != nullptr && choice >= 0 ? choice / p.k : choice;
  return f >= p.T ? -1 : f;
}

// A tile's operands: rows of A (a row number per tile row, clamped) and B.
template <int WM, int WN, int MB, int NB, int S, int FA, int OUT_BF16, int WGRAD>
__global__ void __launch_bounds__(64 * WM * WN, 1) k_moe_gemm(MoeArgs p) {
  constexpr int NW = WM * WN;
  constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN;
  constexpr int SA_ = TM / 8 / NW, SB_ = TN / 8 / NW;  // 8-row slices per wave
  static_assert(TM % (8 * NW) == 0 && TN % (8 * NW) == 0, "whole slices");
  constexpr int SM = (TM + 63) / 64 * 64;  // scale rows of A: by the 64
  static_assert(TN % 64 == 0, "scale rows by the 64");
  constexpr int kStage = (TM + TN) * BK;
  constexpr int kRowB = NB * 64 + 16;  // bytes of a staged output row of a wave, padded
  constexpr int kOut = NW * 16 * kRowB;
  constexpr int kAB = S * kStage > kOut ? S * kStage : kOut;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kAB];
  __shared__ __attribute__((aligned(16))) uint32_t lds_s[S][SM + TN];
  __shared__ int src[TM];  // row of A of each tile row, -1: none

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const View<WGRAD> view{p};
  Place t;
  int L = p.first + int(blockIdx.x);
  Deal deal{0, 0, 0};
  if (!WGRAD) deal = deal_tiles<TM, TN, WGRAD>(p, lane);
  if (!find_place<TM, TN, WGRAD>(p, lane, deal, L, t)) return;
  if (!WGRAD) {
    for (int r = tid; r < TM; r += 64 * NW) src[r] = source_of(p, choice_at(p, t, r));
    __syncthreads();
  }
  auto a_row = [&](int r) {  // row of A of tile row r, always inside A
    if (WGRAD) return min(t.m0 + r, view.rows_a() - 1);
    return max(src[r], 0);
  };
  const int nk = t.nk;

  // ---- loads: lane i of an 8-row slice fills row i / 8, chunk i % 8 of it
  // with the chunk that the swizzle keeps there
  const int lrow = lane >> 3, chunk = 16 * ((lane & 7) ^ lrow);
  const uint8_t *pa[SA_], *pb[SB_];
#pragma unroll
  for (int s = 0; s < SA_; ++s) pa[s] = p.A + int64_t(a_row(8 * (w + NW * s) + lrow)) * view.pitch() + t.k0 + chunk;
#pragma unroll
  for (int s = 0; s < SB_; ++s)
    pb[s] = view.b(t) + int64_t(min(t.n0 + 8 * (w + NW * s) + lrow, view.rows_b() - 1)) * view.pitch() + t.k0 + chunk;
  const uint32_t la = lds_of(lds + 8 * w * BK), lb = lds_of(lds + TM * BK + 8 * w * BK);
  // scales: a step's four bytes of each row; wave w brings 64 rows of A's and
  // then B's (again, where there are fewer rows than lanes, so that every wave
  // has as many loads under way)
  constexpr int SS = (SM + TN) / 64;
  static_assert(SS <= NW, "a wave has one load of scales to a step");
  const int64_t spitch = view.pitch() / 32;
  const int64_t n_sa = int64_t(view.rows_a()) * spitch, n_sb = int64_t(view.rows_b()) * spitch;
  const int sw = w % SS;
  const i32x4 rs = sw < SM / 64 ? rsrc(p.SA, n_sa) : rsrc(view.sb(t), n_sb);
  const int srow = 64 * sw + lane;
  const uint32_t soff = uint32_t(
      (srow < SM ? a_row(min(srow, TM - 1)) : min(t.n0 + srow - SM, view.rows_b() - 1)) * spitch + t.k0 / 32);
  const uint32_t ls = lds_of(reinterpret_cast<const uint8_t*>(&lds_s[0][64 * sw]));
  constexpr int kLoads = SA_ + SB_ + 1;  // of a wave and step
  auto load = [&](int ks, int st) {
#pragma unroll
    for (int s = 0; s < SA_; ++s) dma16(pa[s] + int64_t(ks) * BK, la + uint32_t(st * kStage + 8 * NW * s * BK));
#pragma unroll
    for (int s = 0; s < SB_; ++s) dma16(pb[s] + int64_t(ks) * BK, lb + uint32_t(st * kStage + 8 * NW * s * BK));
    dma4(rs, soff + 4u * uint32_t(ks), ls + uint32_t(st * (SM + TN) * 4));
  };

  const int wm = w % WM, wn = w / WM, g = lane >> 4, r16 = lane & 15;
  const int c0 = 16 * (g ^ (r16 & 7)), c1 = 16 * ((g + 4) ^ (r16 & 7));
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
    const uint8_t* tb = ta + TM * BK;
    const uint32_t* ss = lds_s[st];
    uint32_t qa[MB], qb[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) qa[i] = ss[16 * MB * wm + 16 * i + r16];
#pragma unroll
    for (int j = 0; j < NB; ++j) qb[j] = ss[SM + 16 * NB * wn + 16 * j + r16];
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
    st = st == S - 1 ? 0 : st + 1;
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
    for (int q = 0; q < 16 / RPI; ++q) {
      const int rr = RPI * q + lane / LPR, cc = 4 * (lane % LPR);
      const int tr = 16 * MB * wm + 16 * i + rr;
      const int n = t.n0 + 16 * NB * wn + cc;
      v4f v = *reinterpret_cast<const v4f*>(stg + rr * kRowB + cc * 4);
      if (!WGRAD && src[tr] < 0) v = v4f{0.f, 0.f, 0.f, 0.f};
      if (row_in(t.m0, tr, t.m_end) && n < view.rows_b()) {
        const int64_t o = view.out0(t) + (int64_t(t.m0) + tr) * view.rows_b() + n;
        if (OUT_BF16) {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          __builtin_nontemporal_store(__builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4)),
                                      reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + o));
        } else {
          __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(static_cast<float*>(p.out) + o));
        }
      }
    }
  }
}

// -------------------------------------------------------------- big tiles --
// 256 x 256 by four waves of 128 x 128, one wave per SIMD: a step's LDS reads
// are 128 KiB for 256 MFMAs (eight waves of 64 x 128 read 192 KiB), and the
// accumulators of a wave fill the 256 accumulation registers.  With nothing
// else to run on its SIMD a wave may never wait, so it goes through a step in
// four phases of 16 MFMAs, one for each pairing of the halves of its A and B
// fragments (A0 B0, A0 B1, A1 B1, A1 B0), and reads beside each the half that
// a later phase needs: B1 and A1 of this step, then A0 and B0 of the next
// (B0 fragment by fragment, as its last MFMAs pass).  The reads of a stage end
// in its second phase: the step's one barrier is there, the loads of the step
// after next follow it, and have until the next barrier to land.
//
// A workgroup goes through the tiles blockIdx.x + gridDim.x i.  Between two of
// them the output of the last one goes from the accumulators to memory without
// LDS (lanes exchange halves until each holds 16 neighbouring bytes of a row),
// the loads of the next one's first two steps beside it; the search for the
// one after follows while they land.
template <int FA, int OUT_BF16, int WGRAD, int STREAM_A>
__global__ void __launch_bounds__(256, 1) k_moe_big(MoeArgs p) {
  constexpr int TM = 256, TN = 256, NW = 4;
  constexpr int kStage = (TM + TN) * BK;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds_s[2 * (TM + TN) * 16];
  __shared__ int src[2][TM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = scalar(tid >> 6);
  const View<WGRAD> view{p};
  const Deal deal = deal_tiles<TM, TN, WGRAD>(p, lane);

  // ---- loads: 8 slices of 8 rows of each operand per wave; lane i fills row
  // i / 8, chunk i % 8 of a slice with the chunk that the swizzle keeps there:
  // row r's chunks are XORed with (r / 2) % 8, which puts the chunks that 16
  // rows are read at on 16 different places of the 64 banks.
  // 32-bit offsets from a base that moves on by a step (the launcher sends
  // what they do not reach to k_moe_gemm).
  const int lrow = lane >> 3, chunk = 16 * ((lane & 7) ^ (4 * (w & 1) + (lrow >> 1)));
  const uint8_t *pa, *pb;
  uint32_t off[16];
  const uint32_t lbase = lds_of(lds + 8 * w * BK), ls = lds_of(lds_s + 64 * w * 16);
  uint32_t to = lbase;  // stage that is loaded
  auto load = [&](int s, uint32_t to) {
    const int at = (s < 8 ? 0 : TM * BK) + 8 * NW * (s & 7) * BK;
    if (STREAM_A && s < 8) dma16_stream(pa, off[s], to, at);
    else dma16(s < 8 ? pa : pb, off[s], to, at);
  };
  auto loaded = [&] {  // a whole step
    pa += BK;
    pb += BK;
    to = 2 * lbase + kStage - to;
  };
  // scales: rows 64 w .. of A and of B, four steps (16 bytes) each
  const uint8_t* psb;
  int64_t n_sa, n_sb;
  uint32_t soff[2];
  auto load_scales = [&](int q) {
    dma16(rsrc(p.SA, n_sa), soff[0] + 16u * uint32_t(q), ls + uint32_t((q & 1) * (TM + TN) * 16));
    dma16(rsrc(psb, n_sb), soff[1] + 16u * uint32_t(q), ls + uint32_t((q & 1) * (TM + TN) * 16 + TM * 16));
  };
  // Addresses of tile t, whose rows of A are in src[buf], and its first scales.
  auto begin = [&](const Place& t, int buf) {
    const int m0 = t.m0, n0 = t.n0, nk = t.nk;
    if (nk == 0) return;
    auto a_row = [&](int r) {  // row of A of tile row r, always inside A
      return WGRAD ? min(r, view.rows_a() - 1 - m0) : max(src[buf][r], 0);
    };
    pa = scalar(p.A + t.k0 + (WGRAD ? int64_t(m0) * view.pitch() : 0));
    pb = scalar(view.b(t) + t.k0 + int64_t(n0) * view.pitch());
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = 8 * (w + NW * s) + lrow;
      off[s] = uint32_t(a_row(r)) * uint32_t(view.pitch()) + uint32_t(chunk);
      off[8 + s] = uint32_t(min(r, view.rows_b() - 1 - n0)) * uint32_t(view.pitch()) + uint32_t(chunk);
    }
    const int64_t spitch = view.pitch() / 32;
    psb = view.sb(t);
    n_sa = int64_t(view.rows_a()) * spitch;
    n_sb = int64_t(view.rows_b()) * spitch;
    soff[0] = uint32_t((a_row(64 * w + lane) + (WGRAD ? m0 : 0)) * spitch + t.k0 / 32);
    soff[1] = uint32_t(min(n0 + 64 * w + lane, view.rows_b() - 1) * spitch + t.k0 / 32);
    to = lbase;
    load_scales(0);
  };
  // Quarter q of the loads of a tile's first two steps.
  auto preload = [&](int nk, int q) {
    if (nk <= q / 2) return;
    const uint32_t stage = uint32_t(scalar(int(lbase + (q < 2 ? 0 : kStage))));
#pragma unroll
    for (int s = 0; s < 8; ++s) load(8 * (q & 1) + s, stage);
    if (q & 1) loaded();
  };

  const int wm = w & 1, wn = w >> 1, g = lane >> 4, r16 = lane & 15;
  const int c0 = 16 * (g ^ (r16 >> 1)), c1 = 16 * ((g + 4) ^ (r16 >> 1));
  const int ra = (128 * wm + r16) * BK, rb = (TM + 128 * wn + r16) * BK;
  const int sa = (128 * wm + r16) * 16 + g, sb = (TM + 128 * wn + r16) * 16 + g;
  v4f acc[8][8];  // [column block][row block]
  v8i fa[8], fb[8];
  int qa[8], qb[8];
  int o[4], os[2];  // of the stage that is read: A's two chunks, B's; scales
  auto half = [&](v8i& f, int from, int i) {  // 16 bytes of a fragment
    const uint4 v = *reinterpret_cast<const uint4*>(lds + o[from] + 16 * i * BK);
    const int h = from & 1;
    f[4 * h] = int(v.x);
    f[4 * h + 1] = int(v.y);
    f[4 * h + 2] = int(v.z);
    f[4 * h + 3] = int(v.w);
  };
  auto a_half = [&](int f, int h) { half(fa[f], h, f); };
  auto b_half = [&](int f, int h) { half(fb[f], 2 + h, f); };
  auto a_scale = [&](int f) -> int { return lds_s[os[0] + 16 * 16 * f]; };
  auto b_scale = [&](int f) -> int { return lds_s[os[1] + 16 * 16 * f]; };
  auto next_scales = [&](int ks) {
    os[0] = sa + ((ks >> 2) & 1) * (TM + TN) * 16 + 4 * (ks & 3);
    os[1] = os[0] + sb - sa;
  };
  // In inline asm, for its place among the loads and reads (the compiler
  // moves the builtin past all of them) and for accumulation registers; two
  // wait states first, which an operand that a vector instruction wrote needs.
  auto mfma = [&](int j, int i) {
    if constexpr (FA == 0)
      asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                   : "+a"(acc[j][i])
                   : "v"(fb[j]), "v"(fa[i]), "v"(qb[j]), "v"(qa[i]));
    else
      asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] blgp:1"
                   : "+a"(acc[j][i])
                   : "v"(fb[j]), "v"(fa[i]), "v"(qb[j]), "v"(qa[i]));
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
  // 16 MFMAs of the halves j0 of B and i0 of A, column by column; `beside(x)`
  // comes after the first of each two
  auto phase = [&](int j0, int i0, auto&& beside) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      mfma(j0 + x / 2, i0 + 2 * (x & 1));
      beside(x);
      mfma(j0 + x / 2, i0 + 2 * (x & 1) + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Step ks; LOADS: the step after next follows it, and is loaded.
  auto step = [&](int ks, auto loads) {
    constexpr bool LOADS = decltype(loads)::value;
    phase(0, 0, [&](int x) {
      b_half(4 + x / 2, x & 1);
      if (x & 1) qb[4 + x / 2] = b_scale(4 + x / 2);
    });
    phase(4, 0, [&](int x) {
      a_half(4 + x / 2, x & 1);
      if (x & 1) qa[4 + x / 2] = a_scale(4 + x / 2);
    });
    __builtin_amdgcn_s_waitcnt(vmcnt(0));
    barrier();
    if (LOADS && (ks & 3) == 2) load_scales((ks + 2) >> 2);
    next_scales(ks + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] ^= kStage;
    const uint32_t fill = uint32_t(scalar(int(to)));
    int next[8];  // scales of the next step's A0 and B0
    phase(4, 4, [&](int x) {
      a_half(x / 2, x & 1);
      next[x] = x < 4 ? a_scale(x) : b_scale(x - 4);
      if (LOADS) load(x, fill);
    });
    // fragment f of B0 is free after MFMA 4 f + 3
    phase(0, 4, [&](int x) {
      if (x >= 2) b_half(x / 2 - 1, x & 1);
      if (LOADS) load(8 + x, fill);
    });
    b_half(3, 0);
    b_half(3, 1);
    // in inline asm: as plain copies the bytes would be widened at the head
    // of the next step, after a wait for the reads above
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < 4) asm volatile("v_mov_b32 %0, %1" : "=v"(qa[i]) : "v"(next[i]));
      else asm volatile("v_mov_b32 %0, %1" : "=v"(qb[i - 4]) : "v"(next[i]));
    }
    if (LOADS) loaded();
  };
  // ---- out: lane (g, r16) has columns 4 g .. 4 g + 3 of row r16 of each
  // block.  bfloat16: of two blocks' eight, halves of the wave and then rows
  // of 16 lanes change places until it has columns 8 g .. 8 g + 7 of the 32;
  // then neighbouring rows trade one pair of blocks each, so that a store
  // writes whole 128-byte lines (64 bytes of a row at a time wrote 1.5 times
  // the bytes to memory: 604 against 542 us for 65536 rows, N 4096, K 2048).
  auto output = [&](const Place& t, int buf, auto&& beside) {
    constexpr int kElem = OUT_BF16 ? 2 : 4;
    const int64_t pitch = int64_t(view.rows_b()) * kElem;
    const int n0 = t.n0 + 128 * wn, left = view.rows_b() - n0;  // columns of the wave
    uint8_t* at = static_cast<uint8_t*>(p.out) + view.out0(t) * kElem + byte_at(t.m0, 128 * wm, pitch, n0, kElem);
    const bool odd = r16 & 1;
    uint8_t* const pair = at + (r16 & 14) * pitch + (odd ? 64 : 0) + 16 * g;
    at += r16 * pitch + 16 * g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      beside(i);
      const int tr = 128 * wm + 16 * i + r16;
      const bool none = !WGRAD && src[buf][tr] < 0, in = row_in(t.m0, tr, t.m_end);
      if constexpr (OUT_BF16) {
        const bool even_in = row_in(t.m0, tr & ~1, t.m_end), odd_in = row_in(t.m0, tr | 1, t.m_end);
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // 64 columns
          uint32_t v[2][4];            // 8 columns of 32, twice
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
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
          if (64 * q + (odd ? 32 : 0) + 8 * g < left) {
            uint8_t* const to = pair + 16 * i * pitch + 128 * q;
            if (even_in) __builtin_nontemporal_store(even_row, reinterpret_cast<u32x4_t*>(to));
            if (odd_in) __builtin_nontemporal_store(odd_row, reinterpret_cast<u32x4_t*>(to + pitch));
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
          if (in && 16 * j + 4 * g < left)
            __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(at + 16 * i * pitch + 64 * j));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto publish = [&](const Place& t, int buf, int choice) {  // src[buf] of tile t
    if (WGRAD) return;
    src[buf][tid] = source_of(p, choice);
    __syncthreads();
  };

  Place cur, next{};
  int L = blockIdx.x, buf = 0;
  if (!find_place<TM, TN, WGRAD>(p, lane, deal, L, cur)) return;
  publish(cur, 0, WGRAD ? 0 : choice_at(p, cur, tid));
  begin(cur, 0);
#pragma unroll
  for (int q = 0; q < 4; ++q) preload(cur.nk, q);
  clear();
  for (;;) {
    L += gridDim.x;
    const bool more = find_place<TM, TN, WGRAD>(p, lane, deal, L, next);
    const int choice = WGRAD || !more ? -1 : choice_at(p, next, tid);
    const int nk = cur.nk;
    __builtin_amdgcn_s_waitcnt(vmcnt(0));
    __syncthreads();
    if (nk > 0) {
      o[0] = ra + c0;
      o[1] = ra + c1;
      o[2] = rb + c0;
      o[3] = rb + c1;
      next_scales(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a_half(i, 0);
        a_half(i, 1);
        b_half(i, 0);
        b_half(i, 1);
        qa[i] = a_scale(i);
        qb[i] = b_scale(i);
      }
      settle();  // the zeros, before an MFMA adds to them
      asm volatile("s_nop 15");
      int ks = 0;
      for (; ks < nk - 2; ++ks) step(ks, std::true_type{});
      for (; ks < nk; ++ks) step(ks, std::false_type{});
      asm volatile("s_nop 15\n\ts_nop 15");  // the last MFMAs, before their results are read
      settle();
    }
    // the last step's barrier is past the last reads of both stages that count
    const Place done = cur;
    cur = next;
    if (more) {
      publish(cur, buf ^ 1, choice);
      begin(cur, buf ^ 1);
    }
    const int ahead = more ? cur.nk : 0;
    output(done, buf, [&](int i) {
      if (i < 4) preload(ahead, i);
    });
    if (!more) return;
    buf ^= 1;
    clear();
  }
}

template <int WM, int WN, int MB, int NB, int S, int WGRAD>
bsq_status launch(MoeArgs a, bool e5m2, bool bf16, int64_t grid, hipStream_t st) {
  return in_parts(grid, kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = int(first);
    const dim3 g = dim3(unsigned(n)), b = dim3(64 * WM * WN);
    switch ((e5m2 ? 1 : 0) | (bf16 ? 2 : 0)) {
      case 0: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, S, 0, 0, WGRAD>), g, b, 0, st, a); break;
      case 1: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, S, 1, 0, WGRAD>), g, b, 0, st, a); break;
      case 2: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, S, 0, 1, WGRAD>), g, b, 0, st, a); break;
      default: hipLaunchKernelGGL((k_moe_gemm<WM, WN, MB, NB, S, 1, 1, WGRAD>), g, b, 0, st, a);
    }
    return launch_status(WGRAD ? "moe_wgrad" : "moe_matmul");
  });
}

template <int WGRAD, int STREAM_A>
bsq_status launch_big(const MoeArgs& a, bool e5m2, bool bf16, int64_t grid, hipStream_t st) {
  // one workgroup to a CU, each going through its share of the tiles
  const dim3 g = dim3(unsigned(grid < kCUs ? grid : kCUs)), b = dim3(256);
  switch ((e5m2 ? 1 : 0) | (bf16 ? 2 : 0)) {
    case 0: hipLaunchKernelGGL((k_moe_big<0, 0, WGRAD, STREAM_A>), g, b, 0, st, a); break;
    case 1: hipLaunchKernelGGL((k_moe_big<1, 0, WGRAD, STREAM_A>), g, b, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_moe_big<0, 1, WGRAD, STREAM_A>), g, b, 0, st, a); break;
    default: hipLaunchKernelGGL((k_moe_big<1, 1, WGRAD, STREAM_A>), g, b, 0, st, a);
  }
  return launch_status(WGRAD ? "moe_wgrad" : "moe_matmul");
}

MoeArgs args_of(const MoeGemmLaunch& L) {
  return MoeArgs{L.A, L.B, L.SA, L.SB, L.out, L.offsets, L.rows, L.T, L.cap, L.E, int(L.N), int(L.K), L.k, 0};
}

}  // namespace

bsq_status launch_moe_product(const MoeGemmLaunch& L, hipStream_t st) {
  const MoeArgs a = args_of(L);
  // a segment's last tile may be part full: at most one such tile for each
  // expert and for the rows past the last segment
  auto grid = [&](int tm, int tn) { return (L.cap / tm + L.E + 1) * up_to(L.N, tn); };
  switch (product_tile(L.T, L.cap, L.E, L.N, L.K, L.k, L.rows != nullptr)) {
    case MoeTile::t256x256: return launch_big<0, 0>(a, L.a_e5m2, L.out_bf16, grid(256, 256), st);
    case MoeTile::t32x64: return launch<1, 4, 2, 1, 3, 0>(a, L.a_e5m2, L.out_bf16, grid(32, 64), st);
    case MoeTile::t64x64: return launch<2, 2, 2, 2, 3, 0>(a, L.a_e5m2, L.out_bf16, grid(64, 64), st);
    case MoeTile::t64x128s3: return launch<2, 2, 2, 4, 3, 0>(a, L.a_e5m2, L.out_bf16, grid(64, 128), st);
    default: return launch<2, 2, 2, 4, 2, 0>(a, L.a_e5m2, L.out_bf16, grid(64, 128), st);
  }
}

bsq_status launch_moe_wgrad(const MoeGemmLaunch& L, hipStream_t st) {
  const MoeArgs a = args_of(L);
  auto tiles = [&](int tn, int tk) { return up_to(L.N, tn) * up_to(L.K, tk) * L.E; };
  switch (wgrad_tile(L.cap, L.E, L.N, L.K)) {
    case MoeTile::t256x256_stream: return launch_big<1, 1>(a, L.a_e5m2, L.out_bf16, tiles(256, 256), st);
    case MoeTile::t256x256: return launch_big<1, 0>(a, L.a_e5m2, L.out_bf16, tiles(256, 256), st);
    case MoeTile::t64x64: return launch<2, 2, 2, 2, 3, 1>(a, L.a_e5m2, L.out_bf16, tiles(64, 64), st);
    case MoeTile::t64x128s3: return launch<2, 2, 2, 4, 3, 1>(a, L.a_e5m2, L.out_bf16, tiles(64, 128), st);
    case MoeTile::t128x128s3: return launch<2, 2, 4, 4, 3, 1>(a, L.a_e5m2, L.out_bf16, tiles(128, 128), st);
    default: return launch<2, 2, 4, 4, 2, 1>(a, L.a_e5m2, L.out_bf16, tiles(128, 128), st);
  }
}

}  // namespace bsq
