// The order of an expert layer's rows: sorting the T k choices by expert,
// gathering tokens into 8-bit operands in that order, and summing the
// experts' rows back to their tokens with their weights.
#include "fp8.h"
#include "moe.h"
#include "moe_index.h"

#include <type_traits>

namespace bsq {

namespace {

// ------------------------------------------------------------------- plan --
// A stable counting sort.  Workgroup b owns a contiguous run of choices; the
// row of a choice is its expert's first row, plus the expert's choices in
// earlier workgroups, plus those before it in its own.  Up to kPlanChunk
// choices one workgroup does it all; beyond, a first launch leaves each
// workgroup's counts in `space` and every workgroup of the second sums them
// itself (nothing waits for another workgroup).  No atomic orders anything:
// the result is the same on every run.  65536 choices of 32 experts take 4.6 +
// 6 us (24 in the second launch where one thread summed an expert's counts),
// 128 of 256 experts 4.7 us in one; both are launch and latency.
constexpr int kPlanMaxE = 1024;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int64_t kPlanChunk = 1024;  // choices per workgroup, at least
constexpr int64_t kPlanMaxBlocks = 256;

struct PlanArgs {
  int64_t n, cap;
  int E, align, bits;  // 2^bits >= E
  int64_t chunk;
  const int32_t* ids;
  int32_t *offsets, *counts, *rows, *pos, *space;
};

__global__ void __launch_bounds__(256) k_plan_count(PlanArgs a) {
  __shared__ int hist[kPlanMaxE];
  for (int e = threadIdx.x; e < a.E; e += 256) hist[e] = 0;
  __syncthreads();
  const int64_t begin = int64_t(blockIdx.x) * a.chunk, end = min(begin + a.chunk, a.n);
  for (int64_t i = begin + threadIdx.x; i < end; i += 256) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256) a.space[int64_t(blockIdx.x) * a.E + e] = hist[e];
}

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

template <int ONE>
__global__ void __launch_bounds__(kPlanThreads) k_plan_place(PlanArgs a) {
  extern __shared__ int lds[];
  int* const wcnt = lds;                          // [kPlanWaves][E]
  int* const base = lds + kPlanWaves * a.E;       // [E] next row of each expert in this workgroup
  int64_t* const part_sum = reinterpret_cast<int64_t*>(lds + ((kPlanWaves + 1) * a.E + 1) / 2 * 2);
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int E = a.E, nb = gridDim.x, me = blockIdx.x;
  const int nt = blockDim.x, nw = nt >> 6;
  const int64_t begin = int64_t(me) * a.chunk, end = min(begin + a.chunk, a.n);

  // this workgroup's counts (ONE), else everybody's
  if (ONE) {
    for (int e = tid; e < E; e += nt) base[e] = 0;
    __syncthreads();
    for (int64_t i = begin + tid; i < end; i += nt) {
      const int e = a.ids[i];
      if (e >= 0 && e < E) atomicAdd(&base[e], 1);
    }
    __syncthreads();
  }
  // totals of all workgroups and of the earlier ones: a power of two of
  // threads per expert, each over its share of the workgroups
  int* const sums = lds;  // total [E], before [E]
  int total = 0, before = 0;
  if (ONE) {
    if (tid < E) total = base[tid];
  } else {
    const int x = tid & ((1 << a.bits) - 1), part = tid >> a.bits, parts = nt >> a.bits;
    for (int e = tid; e < 2 * E; e += nt) sums[e] = 0;
    __syncthreads();
    if (x < E) {
      for (int b = part; b < nb; b += parts) {
        const int c = a.space[int64_t(b) * E + x];
        total += c;
        before += b < me ? c : 0;
      }
      atomicAdd(&sums[x], total);
      atomicAdd(&sums[E + x], before);
    }
    __syncthreads();
    total = tid < E ? sums[tid] : 0;
    before = tid < E ? sums[E + tid] : 0;
    __syncthreads();
  }
  // first rows: the sum of the earlier experts' segments
  const int64_t held = tid < E ? (int64_t(total) + a.align - 1) / a.align * a.align : 0;
  const int64_t in = wave_scan(held, lane);
  if (lane == 63) part_sum[w] = in;
  __syncthreads();
  int64_t first = in - held, all = 0;
  for (int v = 0; v < nw; ++v) {
    if (v < w) first += part_sum[v];
    all += part_sum[v];
  }
  int* const hole = lds;  // first and past-the-end row without a choice, of each expert
  if (tid < E) {
    base[tid] = int(first) + before;
    hole[tid] = int(first) + total;
    hole[E + tid] = int(first + held);
    if (me == 0) {
      a.offsets[tid] = int(first);
      a.counts[tid] = total;
      if (tid == E - 1) a.offsets[E] = int(all);
    }
  }
  __syncthreads();
  if (a.align > 1)
    for (int e = me * nw + w; e < E; e += nb * nw)
      for (int64_t r = int64_t(hole[e]) + lane; r < hole[E + e]; r += 64)
        if (r < a.cap) a.rows[r] = -1;
  for (int64_t r = all + int64_t(me) * nt + tid; r < a.cap; r += int64_t(nb) * nt) a.rows[r] = -1;
  __syncthreads();

  for (int64_t i0 = begin; i0 < end; i0 += nt) {
    for (int e = tid; e < nw * E; e += nt) wcnt[e] = 0;
    __syncthreads();
    const int64_t i = i0 + tid;
    int e = i < end ? a.ids[i] : -1;
    if (e < 0 || e >= E) e = -1;
    // the wave's lanes with the same expert
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? set : ~set;
    }
    const int ahead = __popcll(same & ((1ull << lane) - 1ull));
    if (e >= 0 && ahead == 0) wcnt[w * E + e] = __popcll(same);
    __syncthreads();
    for (int x = tid; x < E; x += nt) {
      int at = base[x];
      for (int v = 0; v < nw; ++v) {
        const int c = wcnt[v * E + x];
        wcnt[v * E + x] = at;
        at += c;
      }
      base[x] = at;
    }
    __syncthreads();
    if (i < end) {
      int r = -1;
      if (e >= 0) {
        r = wcnt[w * E + e] + ahead;
        if (r < a.cap) a.rows[r] = int(i);
      }
      a.pos[i] = r;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- gather --
// Rows of x in the experts' order as 8-bit operands: along rows for the
// product, and transposed, in blocks of 32 rows, for the weight gradient.
// A workgroup takes 128 rows x 128 columns; the values go through LDS once,
// so that x is read once for both.  Bfloat16 values without weights stay
// pairs of 16 bits throughout (the hardware converts a pair under a block
// scale in one instruction), else they are float32.  Rows without a choice
// are zeros.
//
// Bound by memory: 16384 tokens of 2048 to 69632 rows, both orientations, read
// 149 MB and write 318 in 75 us, 6.2 TB/s (172 us by 64-column tiles of
// float32).  A token's rows lie k segments apart, so a strip of 128 columns of
// x (4 MB at 16384 tokens) is kept in one XCD's L2 while its tiles are made:
// column strips per XCD 121 us where rows of tiles took 133; non-temporal
// stores, which leave the L2 to x, 88 with them against 121; a scale byte at a
// time instead of words, 15 us more (each of these with the plan's 11 us).
// With weights, or from float32, the tile is of float32 values and 64 KiB, two
// workgroups of 256 threads to a CU: 206 us (bfloat16, e5m2) and 266 (float32)
// for the same rows.
struct GatherArgs {
  int64_t T, H, cap;
  int k;
  const void* x;
  const int32_t* rows;
  const float* weights;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t first;  // tile of this launch
};

template <int SRC_BF16, int PAIRS, int CODE>
__global__ void __launch_bounds__(256) k_gather_mx(GatherArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTile * kTile / (PAIRS ? 2 : 1)];
  __shared__ int src[kTile];
  __shared__ float wt[kTile];
  const int64_t tiles_r = (a.cap + kTile - 1) / kTile;
  const int64_t t = a.first + xcd_run(blockIdx.x, gridDim.x);
  const int64_t r0 = t % tiles_r * kTile, c0 = t / tiles_r * kTile;
  const int tx = threadIdx.x;
  if (tx < kTile) {
    int at = r0 + tx < a.cap ? a.rows[r0 + tx] : -1;
    int from = at >= 0 ? at / a.k : -1;
    if (from >= a.T) from = -1;
    src[tx] = from;
    if (!PAIRS) wt[tx] = from >= 0 && a.weights != nullptr ? a.weights[at] : 1.0f;
  }
  saturate_fp8();
  __syncthreads();
  const int c8 = tx & 15;
  const int64_t c = c0 + 8 * c8;
  const bool words = a.H % kTile == 0 && aligned4(a.scales);
  if constexpr (PAIRS) {
    uint4 v[4][2];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int from = src[2 * ((tx >> 4) + 16 * s) + h];
        v[s][h] = make_uint4(0u, 0u, 0u, 0u);
        if (from >= 0 && c < a.H)
          v[s][h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + from * a.H + c);
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int rp = (tx >> 4) + 16 * s;
      const uint32_t lo[4] = {v[s][0].x, v[s][0].y, v[s][0].z, v[s][0].w};
      const uint32_t hi[4] = {v[s][1].x, v[s][1].y, v[s][1].z, v[s][1].w};
      const int64_t r = r0 + 2 * rp;
      if (a.codes != nullptr) {
        put_row<CODE>(a.codes, a.scales, (r * a.H + c) / 8, r < a.cap && c < a.H, words, lo);
        put_row<CODE>(a.codes, a.scales, ((r + 1) * a.H + c) / 8, r + 1 < a.cap && c < a.H, words, hi);
      }
      if (a.codes_t != nullptr) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[2 * i] = __builtin_amdgcn_perm(hi[i], lo[i], 0x05040100u);      // column 2 i of both rows
          w[2 * i + 1] = __builtin_amdgcn_perm(hi[i], lo[i], 0x07060302u);  // column 2 i + 1
        }
        uint4* o = reinterpret_cast<uint4*>(tile + tile_at<1>(rp, c8));
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int rr = (tx >> 4) + 16 * s;
      const int64_t r = r0 + rr;
      const int from = src[rr];
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (from >= 0 && c < a.H) {
        load8<SRC_BF16>(a.x, from * a.H + c, x);
        if (a.weights != nullptr) {
          const float f = wt[rr];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= f;
        }
      }
      if (a.codes != nullptr) put_row<CODE>(a.codes, a.scales, (r * a.H + c) / 8, r < a.cap && c < a.H, words, x);
      if (a.codes_t != nullptr) {
        float4* o = reinterpret_cast<float4*>(tile + tile_at<0>(rr, c8));
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  }
  if (a.codes_t == nullptr) return;
  __syncthreads();
  put_columns<CODE, PAIRS, 256>(tile, r0, c0, a.cap, a.H, a.codes_t, a.scales_t);
}

// ---------------------------------------------------------------- combine --
// out[t] = sum over j of weights[t, j] y[pos[t, j]], in float32 in the order
// of j; a choice without a row (pos < 0) adds nothing.  Eight columns per
// thread.  Bound by the one read of y: 8192 tokens, 8 rows each of 2048, 302
// MB in 59 us (5.1 TB/s), its gradient 302 MB in 63 us.
struct CombineArgs {
  int64_t T, H, cap;
  int k;
  const void* y;
  const int32_t* pos;
  const float* weights;
  const void* dout;
  void* out;  // combine: out; its gradient: dweights
};

template <int BF16>
__global__ void __launch_bounds__(256) k_combine(CombineArgs a) {
  const int64_t h8 = a.H / 8, n = a.T * h8;
  for (int64_t f = int64_t(blockIdx.x) * 256 + threadIdx.x; f < n; f += int64_t(gridDim.x) * 256) {
    const int64_t t = f / h8, c = (f - t * h8) * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = a.pos[t * a.k + j];
      if (r < 0 || r >= a.cap) continue;
      const float wt = a.weights != nullptr ? a.weights[t * a.k + j] : 1.0f;
      float y[8];
      load8<BF16>(a.y, r * a.H + c, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = fmaf(wt, y[i], s[i]);
    }
    store8<BF16>(a.out, t * a.H + c, s);
  }
}

// dweights[t, j] = y[pos[t, j]] . dout[t], one wave per token; kBatch choices
// at a time, so that dout is read once for them and their rows' loads are all
// under way together.
constexpr int kBatch = 8;
template <int BF16>
__global__ void __launch_bounds__(256) k_combine_backward(CombineArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    int64_t row[kBatch];
    float s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = j0 + j < a.k ? a.pos[t * a.k + j0 + j] : -1;
      row[j] = r >= 0 && r < a.cap ? int64_t(r) : -1;
      s[j] = 0.f;
    }
    for (int64_t c = lane * 8; c < a.H; c += 512) {
      float d[8], y[kBatch][8];
      load8<BF16>(a.dout, t * a.H + c, d);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (row[j] >= 0) load8<BF16>(a.y, row[j] * a.H + c, y[j]);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (row[j] >= 0)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[j] = fmaf(y[j][i], d[i], s[j]);
    }
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) s[j] += __shfl_xor(s[j], m);
      if (lane == j) mine = s[j];
    }
    if (lane < kBatch && j0 + lane < a.k) static_cast<float*>(a.out)[t * a.k + j0 + lane] = mine;
  }
}

}  // namespace

int plan_blocks(int64_t n) {
  const int64_t b = (n + kPlanChunk - 1) / kPlanChunk;
  return int(b < 1 ? 1 : (b < kPlanMaxBlocks ? b : kPlanMaxBlocks));
}

bsq_status launch_plan(int64_t n, int E, int align, int64_t cap, const int32_t* ids, int32_t* offsets,
                       int32_t* counts, int32_t* rows, int32_t* pos, int32_t* space, hipStream_t st) {
  PlanArgs a{n, cap, E, align, 0, 0, ids, offsets, counts, rows, pos, space};
  while ((1 << a.bits) < E) ++a.bits;
  const int nb = plan_blocks(n);
  a.chunk = nb == 1 ? n : (n + nb - 1) / nb;
  const size_t lds = size_t((kPlanWaves + 1) * E + 2) * 4 + kPlanWaves * 8;
  if (nb == 1) {
    hipLaunchKernelGGL(k_plan_place<1>, 1, kPlanThreads, lds, st, a);
  } else {
    hipLaunchKernelGGL(k_plan_count, nb, 256, 0, st, a);
    hipLaunchKernelGGL(k_plan_place<0>, nb, kPlanThreads, lds, st, a);
  }
  return launch_status("moe_plan");
}

bsq_status launch_gather_mx(int64_t T, int64_t H, int64_t cap, int k, const void* x, bool bf16, const int32_t* rows,
                            const float* weights, bool e5m2, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                            uint8_t* scales_t, hipStream_t st) {
  GatherArgs a{T, H, cap, k, x, rows, weights, codes, scales, codes_t, scales_t, 0};
  const int form = !bf16 ? 0 : weights != nullptr ? 1 : 2;
  return in_parts(((cap + kTile - 1) / kTile) * ((H + kTile - 1) / kTile), kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = first;
    const unsigned grid = unsigned(n);
    switch (form | (e5m2 ? 4 : 0)) {
      case 0: hipLaunchKernelGGL((k_gather_mx<0, 0, 0>), grid, 256, 0, st, a); break;
      case 1: hipLaunchKernelGGL((k_gather_mx<1, 0, 0>), grid, 256, 0, st, a); break;
      case 2: hipLaunchKernelGGL((k_gather_mx<1, 1, 0>), grid, 256, 0, st, a); break;
      case 4: hipLaunchKernelGGL((k_gather_mx<0, 0, 1>), grid, 256, 0, st, a); break;
      case 5: hipLaunchKernelGGL((k_gather_mx<1, 0, 1>), grid, 256, 0, st, a); break;
      default: hipLaunchKernelGGL((k_gather_mx<1, 1, 1>), grid, 256, 0, st, a);
    }
    return launch_status("moe_gather_mx");
  });
}

bsq_status launch_combine(int64_t T, int64_t H, int64_t cap, int k, const void* y, bool bf16, const int32_t* pos,
                          const float* weights, void* out, hipStream_t st) {
  const CombineArgs a{T, H, cap, k, y, pos, weights, nullptr, out};
  const int64_t want = (T * (H / 8) + 255) / 256;
  const unsigned grid = unsigned(want < (1 << 20) ? want : (1 << 20));
  if (bf16) hipLaunchKernelGGL(k_combine<1>, grid, 256, 0, st, a);
  else hipLaunchKernelGGL(k_combine<0>, grid, 256, 0, st, a);
  return launch_status("moe_combine");
}

bsq_status launch_combine_backward(int64_t T, int64_t H, int64_t cap, int k, const void* y, bool bf16,
                                   const int32_t* pos, const void* dout, float* dweights, hipStream_t st) {
  return in_parts(T, kLaunchTokens, [&](int64_t t, int64_t n) {
    const CombineArgs a{n, H, cap, k, y, pos + t * k, nullptr,
                        static_cast<const char*>(dout) + t * H * (bf16 ? 2 : 4), dweights + t * k};
    const unsigned grid = unsigned((n + 3) / 4);
    if (bf16) hipLaunchKernelGGL(k_combine_backward<1>, grid, 256, 0, st, a);
    else hipLaunchKernelGGL(k_combine_backward<0>, grid, 256, 0, st, a);
    return launch_status("moe_combine_backward");
  });
}

}  // namespace bsq
