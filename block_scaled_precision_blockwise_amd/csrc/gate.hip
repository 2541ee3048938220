// The gated activation between an expert's two products, with its 8-bit
// checkpoint: h = g sigmoid(g) u of gu = [g | u], quantized along rows (the
// next product's operand) and, for training, down columns (the weight
// gradient's operand), and g and u themselves in 8 bits, from which the
// backward pass takes its gradient instead of from 16-bit copies.
#include "fp8.h"
#include "moe.h"

namespace bsq {

namespace {

constexpr int kTR = 128, kTC = 64;

// 1 / (1 + e^-g) in float32; e^-g = inf gives 0.
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

struct GateArgs {
  int64_t R, F;
  const void* gu;
  uint8_t *h, *hs, *ht, *hts, *kept, *kepts;
};

template <int CODE>
__device__ __forceinline__ void put_row8(uint8_t* codes, uint8_t* scales, int64_t f8, const float (&x)[8], bool in) {
  constexpr int EMAX = CODE == 0 ? 8 : 15;
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
  const int E = mx_exponent<EMAX>(__uint_as_float(group_max_bits<4>(m)));
  if (!in) return;
  reinterpret_cast<uint2*>(codes)[f8] = make_uint2(mx_encode4<CODE>(&x[0], E), mx_encode4<CODE>(&x[4], E));
  if ((f8 & 3) == 0) scales[f8 >> 2] = uint8_t(E + 127);
}

template <int SRC_BF16, int CODE>
__global__ void __launch_bounds__(256) k_swiglu_mx(GateArgs a) {
  constexpr int EMAX = CODE == 0 ? 8 : 15;
  __shared__ float tile[kTR][kTC + 1];
  const int64_t tiles_c = (a.F + kTC - 1) / kTC;
  const int64_t r0 = int64_t(blockIdx.x) / tiles_c * kTR, c0 = int64_t(blockIdx.x) % tiles_c * kTC;
  const int tx = threadIdx.x;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = (tx >> 3) + 32 * s, cg = (tx & 7) * 8;
    const bool in = r0 + r < a.R && c0 + cg < a.F;
    float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int64_t at = (r0 + r) * 2 * a.F + c0 + cg;
    if (in) {
      load8<SRC_BF16>(a.gu, at, g);
      load8<SRC_BF16>(a.gu, at + a.F, u);
    }
    if (a.kept != nullptr) {
      put_row8<CODE>(a.kept, a.kepts, at / 8, g, in);
      put_row8<CODE>(a.kept, a.kepts, (at + a.F) / 8, u, in);
    }
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
    put_row8<CODE>(a.h, a.hs, ((r0 + r) * a.F + c0 + cg) / 8, h, in);
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[r][cg + i] = h[i];
  }
  if (a.ht == nullptr) return;
  __syncthreads();
  const int oc = tx >> 2, seg = tx & 3;
  const int64_t r = r0 + 32 * seg, c = c0 + oc;
  if (r >= a.R || c >= a.F) return;
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
  uint4* o = reinterpret_cast<uint4*>(a.ht + c * a.R + r);
  o[0] = make_uint4(q[0], q[1], q[2], q[3]);
  o[1] = make_uint4(q[4], q[5], q[6], q[7]);
  a.hts[c * (a.R / 32) + r / 32] = uint8_t(E + 127);
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
    store8<BF16>(a.dgu, gi * 8, dg);
    store8<BF16>(a.dgu, ui * 8, du);
  }
}

}  // namespace

bsq_status launch_swiglu_mx(int64_t R, int64_t F, const void* gu, bool bf16, bool e5m2, uint8_t* h, uint8_t* h_scales,
                            uint8_t* ht, uint8_t* ht_scales, uint8_t* kept, uint8_t* kept_scales, hipStream_t st) {
  const GateArgs a{R, F, gu, h, h_scales, ht, ht_scales, kept, kept_scales};
  const unsigned grid = unsigned(((R + kTR - 1) / kTR) * ((F + kTC - 1) / kTC));
  switch ((bf16 ? 1 : 0) | (e5m2 ? 2 : 0)) {
    case 0: hipLaunchKernelGGL((k_swiglu_mx<0, 0>), grid, 256, 0, st, a); break;
    case 1: hipLaunchKernelGGL((k_swiglu_mx<1, 0>), grid, 256, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_swiglu_mx<0, 1>), grid, 256, 0, st, a); break;
    default: hipLaunchKernelGGL((k_swiglu_mx<1, 1>), grid, 256, 0, st, a);
  }
  return launch_status("swiglu_mx");
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
