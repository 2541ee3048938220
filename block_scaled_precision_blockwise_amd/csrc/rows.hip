// The order of an expert layer's rows: sorting the T k choices by expert,
// gathering tokens into 8-bit operands in that order, and summing the
// experts' rows back to their tokens with their weights.
#include "fp8.h"
#include "moe.h"

#include <type_traits>

namespace bsq {

namespace {

// ------------------------------------------------------------------- plan --
// A stable counting sort.  Workgroup b owns a contiguous run of choices; the
// row of a choice is its expert's first row, plus the expert's choices in
// earlier workgroups, plus those before it in its own.  Up to kPlanOne
// choices one workgroup does it all; beyond, a first launch leaves each
// workgroup's counts in `space` and every workgroup of the second sums them
// itself (nothing waits for another workgroup).  No atomic orders anything:
// the result is the same on every run.
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
  int64_t* const part = reinterpret_cast<int64_t*>(lds + ((kPlanWaves + 1) * a.E + 1) / 2 * 2);  // [kPlanWaves]
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
  int total = 0, before = 0;
  if (tid < E) {
    if (ONE) {
      total = base[tid];
    } else {
      for (int b = 0; b < nb; ++b) {
        const int c = a.space[int64_t(b) * E + tid];
        total += c;
        before += b < me ? c : 0;
      }
    }
  }
  // first rows: the sum of the earlier experts' segments
  const int64_t held = tid < E ? (int64_t(total) + a.align - 1) / a.align * a.align : 0;
  const int64_t in = wave_scan(held, lane);
  if (lane == 63) part[w] = in;
  __syncthreads();
  int64_t first = in - held, all = 0;
  for (int v = 0; v < nw; ++v) {
    if (v < w) first += part[v];
    all += part[v];
  }
  if (tid < E) {
    base[tid] = int(first) + before;
    if (me == 0) {
      a.offsets[tid] = int(first);
      a.counts[tid] = total;
      if (tid == E - 1) a.offsets[E] = int(all);
    }
    // the segment's rows without a choice
    if (tid % nb == me)
      for (int64_t r = first + total; r < first + held; ++r)
        if (r < a.cap) a.rows[r] = -1;
  }
  for (int64_t r = all + int64_t(me) * nt + tid; r < a.cap; r += int64_t(nb) * nt) a.rows[r] = -1;

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
// A workgroup takes 128 rows x 64 columns; the values go through LDS once,
// so that x is read once for both and a line of the transposed codes is
// written whole.  Rows without a choice are zeros.
constexpr int kTR = 128, kTC = 64;

// One 32-row block of a column per thread: codes and scale of rows
// r0 + 32 seg .. + 31 of column c0 + oc, transposed.
template <int CODE>
__device__ __forceinline__ void put_transposed(const float (*tile)[kTC + 1], int64_t r0, int64_t c0, int64_t rows,
                                               int64_t cols, uint8_t* codes_t, uint8_t* scales_t) {
  constexpr int EMAX = CODE == 0 ? 8 : 15;
  const int oc = threadIdx.x >> 2, seg = threadIdx.x & 3;
  const int64_t r = r0 + 32 * seg, c = c0 + oc;
  if (r >= rows || c >= cols) return;
  float x[32];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    x[i] = tile[32 * seg + i][oc];
    m = max(m, abs_bits(x[i]));
  }
  const int E = mx_exponent<EMAX>(__uint_as_float(m));
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = mx_encode4<CODE>(&x[4 * i], E);
  uint4* o = reinterpret_cast<uint4*>(codes_t + c * rows + r);
  o[0] = make_uint4(q[0], q[1], q[2], q[3]);
  o[1] = make_uint4(q[4], q[5], q[6], q[7]);
  scales_t[c * (rows / 32) + r / 32] = uint8_t(E + 127);
}

struct GatherArgs {
  int64_t T, H, cap;
  int k;
  const void* x;
  const int32_t* rows;
  const float* weights;
  uint8_t *codes, *scales, *codes_t, *scales_t;
};

template <int SRC_BF16, int CODE>
__global__ void __launch_bounds__(256) k_gather_mx(GatherArgs a) {
  constexpr int EMAX = CODE == 0 ? 8 : 15;
  __shared__ float tile[kTR][kTC + 1];
  const int64_t tiles_c = (a.H + kTC - 1) / kTC;
  const int64_t r0 = int64_t(blockIdx.x) / tiles_c * kTR, c0 = int64_t(blockIdx.x) % tiles_c * kTC;
  const int tx = threadIdx.x;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = (tx >> 3) + 32 * s, cg = (tx & 7) * 8;
    const bool in = r0 + r < a.cap && c0 + cg < a.H;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int at = in ? a.rows[r0 + r] : -1;
    const int64_t t = at >= 0 ? at / a.k : a.T;
    if (t < a.T) {
      load8<SRC_BF16>(a.x, t * a.H + c0 + cg, x);
      if (a.weights != nullptr) {
        const float wt = a.weights[at];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= wt;
      }
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
    const int E = mx_exponent<EMAX>(__uint_as_float(group_max_bits<4>(m)));
    if (in && a.codes != nullptr) {
      const int64_t f = ((r0 + r) * a.H + c0 + cg) / 8;
      reinterpret_cast<uint2*>(a.codes)[f] = make_uint2(mx_encode4<CODE>(&x[0], E), mx_encode4<CODE>(&x[4], E));
      if ((tx & 3) == 0) a.scales[f >> 2] = uint8_t(E + 127);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[r][cg + i] = x[i];
  }
  if (a.codes_t == nullptr) return;
  __syncthreads();
  put_transposed<CODE>(tile, r0, c0, a.cap, a.H, a.codes_t, a.scales_t);
}

// ---------------------------------------------------------------- combine --
// out[t] = sum over j of weights[t, j] y[pos[t, j]], in float32 in the order
// of j; a choice without a row (pos < 0) adds nothing.  Eight columns per
// thread.
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

// dweights[t, j] = y[pos[t, j]] . dout[t], one wave per token.
template <int BF16>
__global__ void __launch_bounds__(256) k_combine_backward(CombineArgs a) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); t < a.T; t += int64_t(gridDim.x) * 4) {
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = a.pos[t * a.k + j];
      float s = 0.f;
      if (r >= 0 && r < a.cap) {
        for (int64_t c = lane * 8; c < a.H; c += 512) {
          float y[8], d[8];
          load8<BF16>(a.y, r * a.H + c, y);
          load8<BF16>(a.dout, t * a.H + c, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) s = fmaf(y[i], d[i], s);
        }
      }
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
      if (lane == 0) static_cast<float*>(a.out)[t * a.k + j] = s;
    }
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
  const GatherArgs a{T, H, cap, k, x, rows, weights, codes, scales, codes_t, scales_t};
  const unsigned grid = unsigned(((cap + kTR - 1) / kTR) * ((H + kTC - 1) / kTC));
  switch ((bf16 ? 1 : 0) | (e5m2 ? 2 : 0)) {
    case 0: hipLaunchKernelGGL((k_gather_mx<0, 0>), grid, 256, 0, st, a); break;
    case 1: hipLaunchKernelGGL((k_gather_mx<1, 0>), grid, 256, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_gather_mx<0, 1>), grid, 256, 0, st, a); break;
    default: hipLaunchKernelGGL((k_gather_mx<1, 1>), grid, 256, 0, st, a);
  }
  return launch_status("moe_gather_mx");
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
  const CombineArgs a{T, H, cap, k, y, pos, nullptr, dout, dweights};
  const int64_t want = (T + 3) / 4;
  const unsigned grid = unsigned(want < (1 << 20) ? want : (1 << 20));
  if (bf16) hipLaunchKernelGGL(k_combine_backward<1>, grid, 256, 0, st, a);
  else hipLaunchKernelGGL(k_combine_backward<0>, grid, 256, 0, st, a);
  return launch_status("moe_combine_backward");
}

}  // namespace bsq
