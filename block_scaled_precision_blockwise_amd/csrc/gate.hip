// The gated activation between an expert's two products, with its 8-bit
// checkpoint: h = g sigmoid(g) u of gu = [g | u], quantized along rows (the
// next product's operand) and, for training, down columns (the weight
// gradient's operand), and g and u themselves in 8 bits, from which the
// backward pass takes its gradient instead of from 16-bit copies.
//
// A stream: 32768 x 2048 reads 268 MB and writes 277 (forward, 114 us) and
// reads 272 and writes 268 (backward, 84 us); the two calls take 198 us, 5.4
// TB/s, the rate of a large copy.  What it took: g and u as pairs of 16 bits
// to the conversion that scales, tiles of 128 columns so that codes are
// written in whole lines both ways, non-temporal stores, and a sigmoid of 10
// instructions; with the library's, single conversions and 64-column tiles it
// was bound by instruction issue (245 us).
#include "fp8.h"
#include "moe.h"
#include "moe_index.h"

#include <type_traits>

namespace bsq {

namespace {

// 1 / (1 + e^-g) in float32 within 4 steps of 2^-23: -g log2 e in two pieces
// (the hardware's 2^t of the first, times 1 + ln 2 of the second), and the
// hardware's reciprocal, of a sixteenth of the sum so that a result near
// 2^-126 is not flushed.  e^-g = inf gives 0.  10 instructions; the library's
// expf and division took 40, and with them the training pass was bound by
// instruction issue.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f;  // log2 e = kLog2e + kRest
  g = __builtin_amdgcn_fmed3f(g, -128.f, 128.f);  // 0 and 1 from there on; keeps infinities out of `lo`
  const float t = -g * kLog2e;
  const float lo = fmaf(-g, kRest, fmaf(-g, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(lo, 0x1.62e43p-1f, 1.0f);
  return __builtin_amdgcn_rcpf(fmaf(e, 0.0625f, 0.0625f)) * 0.0625f;
}

struct GateArgs {
  int64_t R, F;
  const void* gu;
  uint8_t *h, *hs, *ht, *hts, *kept, *kepts;
  int64_t first;  // workgroup or tile of this launch
};

// Eight columns of g, from element `at` of gu, and of u as loaded (zeros where
// not `in`).
template <int SRC_BF16>
struct Raw {
  uint4 g[SRC_BF16 ? 1 : 2], u[SRC_BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const GateArgs& a, int64_t at, bool in) {
#pragma unroll
    for (int i = 0; i < (SRC_BF16 ? 1 : 2); ++i) {
      g[i] = u[i] = make_uint4(0u, 0u, 0u, 0u);
      if (in) {
        const char* p = static_cast<const char*>(a.gu) + at * (SRC_BF16 ? 2 : 4) + 16 * i;
        g[i] = ldnt(reinterpret_cast<const uint4*>(p));
        u[i] = ldnt(reinterpret_cast<const uint4*>(p + a.F * (SRC_BF16 ? 2 : 4)));
      }
    }
  }
};
__device__ __forceinline__ void widen(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = decode_bf16(w[i] & 0xFFFFu);
    x[2 * i + 1] = decode_bf16(w[i] >> 16);
  }
}

// Writes the checkpoint's codes of those columns and, from element `out` on,
// h's, 16 lanes to 128 columns, and leaves h in x.
template <int SRC_BF16, int CODE>
__device__ __forceinline__ void gate8(const GateArgs& a, const Raw<SRC_BF16>& raw, int64_t at, int64_t out,
                                      bool in, bool words, float (&x)[8]) {
  float g[8], u[8];
  if constexpr (SRC_BF16) {
    const uint32_t gw[4] = {raw.g[0].x, raw.g[0].y, raw.g[0].z, raw.g[0].w};
    const uint32_t uw[4] = {raw.u[0].x, raw.u[0].y, raw.u[0].z, raw.u[0].w};
    if (a.kept != nullptr) {
      put_row<CODE>(a.kept, a.kepts, at / 8, in, words, gw);
      put_row<CODE>(a.kept, a.kepts, (at + a.F) / 8, in, words, uw);
    }
    widen(gw, g);
    widen(uw, u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 &gq = raw.g[i / 4], &uq = raw.u[i / 4];
      g[i] = __uint_as_float(i % 4 == 0 ? gq.x : i % 4 == 1 ? gq.y : i % 4 == 2 ? gq.z : gq.w);
      u[i] = __uint_as_float(i % 4 == 0 ? uq.x : i % 4 == 1 ? uq.y : i % 4 == 2 ? uq.z : uq.w);
    }
    if (a.kept != nullptr) {
      put_row<CODE>(a.kept, a.kepts, at / 8, in, words, g);
      put_row<CODE>(a.kept, a.kepts, (at + a.F) / 8, in, words, u);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = g[i] * sigmoid(g[i]) * u[i];
  put_row<CODE>(a.h, a.hs, out / 8, in, words, x);
}

// Without the transposed operand: a stream of rows, eight columns per thread.
template <int SRC_BF16, int CODE>
__global__ void __launch_bounds__(256) k_swiglu_mx_rows(GateArgs a) {
  saturate_fp8();
  const int64_t f8 = a.F / 8, f = (a.first + blockIdx.x) * 256 + threadIdx.x;
  const bool in = f < a.R * f8, words = a.F % kTile == 0 && aligned4(a.hs) && aligned4(a.kepts);
  const int64_t r = in ? f / f8 : 0, c = in ? (f - r * f8) * 8 : 0;
  Raw<SRC_BF16> raw;
  raw.load(a, r * 2 * a.F + c, in);
  float x[8];
  gate8<SRC_BF16, CODE>(a, raw, r * 2 * a.F + c, r * a.F + c, in, words, x);
}

// Eight waves to a tile: 200 us forward and backward, four 202, sixteen 200.
constexpr int kThreads = 512;
template <int SRC_BF16, int CODE>
__global__ void __launch_bounds__(kThreads) k_swiglu_mx(GateArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTile * kTile];
  const int64_t tiles_c = (a.F + kTile - 1) / kTile;
  const int64_t t = a.first + xcd_run(blockIdx.x, gridDim.x);
  const int64_t r0 = t / tiles_c * kTile, c0 = t % tiles_c * kTile;
  const int tx = threadIdx.x, c8 = tx & 15;
  const int64_t c = c0 + 8 * c8;
  const bool words = a.F % kTile == 0 && aligned4(a.hs) && aligned4(a.kepts);
  saturate_fp8();
  // every load first: 64 KiB of LDS leave two workgroups to a CU, so each
  // has to keep its whole tile under way
  constexpr int kRows = kTile * 16 / kThreads;  // rows of a thread
  constexpr int kAhead = SRC_BF16 ? kRows : kRows / 2;
  const int64_t out0 = (r0 + (tx >> 4)) * a.F + c, at0 = 2 * out0 - c;
  auto rows = [&](auto whole) {  // whole: no column or row of the tile is outside
    constexpr bool kWhole = decltype(whole)::value;
    for (int s0 = 0; s0 < kRows; s0 += kAhead) {
      Raw<SRC_BF16> raw[kAhead];
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int rr = (tx >> 4) + kThreads / 16 * (s0 + s);
        raw[s].load(a, at0 + kThreads / 8 * (s0 + s) * a.F, kWhole || (r0 + rr < a.R && c < a.F));
      }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int rr = (tx >> 4) + kThreads / 16 * (s0 + s);
        float x[8];
        gate8<SRC_BF16, CODE>(a, raw[s], at0 + kThreads / 8 * (s0 + s) * a.F, out0 + kThreads / 16 * (s0 + s) * a.F,
                              kWhole || (r0 + rr < a.R && c < a.F), words, x);
        float4* o = reinterpret_cast<float4*>(tile + tile_at<0>(rr, c8));
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  };
  if (r0 + kTile <= a.R && c0 + kTile <= a.F) rows(std::true_type{});
  else rows(std::false_type{});
  __syncthreads();
  put_columns<CODE, 0, kThreads>(tile, r0, c0, a.R, a.F, a.ht, a.hts);
}

// ------------------------------------------------------------- gradient --
struct GateBwdArgs {
  int64_t R, F;
  const uint8_t *kept, *kepts;
  const void* dh;
  void* dgu;
};

template <int CODE>
__device__ __forceinline__ void decode8(uint2 q, int E, float (&v)[8]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int b = int(w == 0 ? q.x : q.y);
    const auto lo = CODE == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8(b, false) : __builtin_amdgcn_cvt_pk_f32_bf8(b, false);
    const auto hi = CODE == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8(b, true) : __builtin_amdgcn_cvt_pk_f32_bf8(b, true);
    v[4 * w] = ldexpf(lo[0], E);
    v[4 * w + 1] = ldexpf(lo[1], E);
    v[4 * w + 2] = ldexpf(hi[0], E);
    v[4 * w + 3] = ldexpf(hi[1], E);
  }
}

// With s = sigmoid(g): dg = dh u s (1 + g (1 - s)), du = dh g s.
template <int BF16, int CODE>
__global__ void __launch_bounds__(256) k_swiglu_mx_backward(GateBwdArgs a) {
  const int64_t f8 = a.F / 8, n = a.R * f8;
  for (int64_t f = int64_t(blockIdx.x) * 256 + threadIdx.x; f < n; f += int64_t(gridDim.x) * 256) {
    const int64_t r = f / f8, c = f - r * f8;  // 8 columns from 8 c
    const int64_t gi = r * 2 * f8 + c, ui = gi + f8;
    float g[8], u[8], dh[8], dg[8], du[8];
    decode8<CODE>(reinterpret_cast<const uint2*>(a.kept)[gi], int(a.kepts[gi >> 2]) - 127, g);
    decode8<CODE>(reinterpret_cast<const uint2*>(a.kept)[ui], int(a.kepts[ui >> 2]) - 127, u);
    load8<BF16>(a.dh, f * 8, dh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      du[i] = dh[i] * g[i] * s;
      dg[i] = dh[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
    }
    store8nt<BF16>(a.dgu, gi * 8, dg);
    store8nt<BF16>(a.dgu, ui * 8, du);
  }
}

}  // namespace

bsq_status launch_swiglu_mx(int64_t R, int64_t F, const void* gu, bool bf16, bool e5m2, uint8_t* h, uint8_t* h_scales,
                            uint8_t* ht, uint8_t* ht_scales, uint8_t* kept, uint8_t* kept_scales, hipStream_t st) {
  const int form = (bf16 ? 1 : 0) | (e5m2 ? 2 : 0);
  GateArgs a{R, F, gu, h, h_scales, ht, ht_scales, kept, kept_scales, 0};
  if (ht == nullptr) {
    return in_parts((R * (F / 8) + 255) / 256, kLaunchGroups, [&](int64_t first, int64_t n) {
      a.first = first;
      const unsigned grid = unsigned(n);
      switch (form) {
        case 0: hipLaunchKernelGGL((k_swiglu_mx_rows<0, 0>), grid, 256, 0, st, a); break;
        case 1: hipLaunchKernelGGL((k_swiglu_mx_rows<1, 0>), grid, 256, 0, st, a); break;
        case 2: hipLaunchKernelGGL((k_swiglu_mx_rows<0, 1>), grid, 256, 0, st, a); break;
        default: hipLaunchKernelGGL((k_swiglu_mx_rows<1, 1>), grid, 256, 0, st, a);
      }
      return launch_status("swiglu_mx");
    });
  }
  return in_parts(((R + kTile - 1) / kTile) * ((F + kTile - 1) / kTile), kLaunchGroups, [&](int64_t first, int64_t n) {
    a.first = first;
    const unsigned grid = unsigned(n);
    switch (form) {
      case 0: hipLaunchKernelGGL((k_swiglu_mx<0, 0>), grid, kThreads, 0, st, a); break;
      case 1: hipLaunchKernelGGL((k_swiglu_mx<1, 0>), grid, kThreads, 0, st, a); break;
      case 2: hipLaunchKernelGGL((k_swiglu_mx<0, 1>), grid, kThreads, 0, st, a); break;
      default: hipLaunchKernelGGL((k_swiglu_mx<1, 1>), grid, kThreads, 0, st, a);
    }
    return launch_status("swiglu_mx");
  });
}

bsq_status launch_swiglu_mx_backward(int64_t R, int64_t F, const uint8_t* kept, const uint8_t* kept_scales, bool e5m2,
                                     const void* dh, bool bf16, void* dgu, hipStream_t st) {
  const GateBwdArgs a{R, F, kept, kept_scales, dh, dgu};
  const int64_t want = (R * (F / 8) + 255) / 256;
  const unsigned grid = unsigned(want < (1 << 20) ? want : (1 << 20));
  switch ((bf16 ? 1 : 0) | (e5m2 ? 2 : 0)) {
    case 0: hipLaunchKernelGGL((k_swiglu_mx_backward<0, 0>), grid, 256, 0, st, a); break;
    case 1: hipLaunchKernelGGL((k_swiglu_mx_backward<1, 0>), grid, 256, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_swiglu_mx_backward<0, 1>), grid, 256, 0, st, a); break;
    default: hipLaunchKernelGGL((k_swiglu_mx_backward<1, 1>), grid, 256, 0, st, a);
  }
  return launch_status("swiglu_mx_backward");
}

}  // namespace bsq
