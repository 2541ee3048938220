// Device helpers of the kernels that write fp8 blocks: block maxima across
// lanes, the E8M0 exponent rule, the fp8 conversions and 8-value loads.
#pragma once

#include "common.h"

namespace bsq {

constexpr float kE4M3Max = 448.0f;
constexpr float kE5M2Max = 57344.0f;

// |x| as bits: for finite x the unsigned order of these is the order of |x|.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t amax4_bits(float4 v) {
  return max(max(abs_bits(v.x), abs_bits(v.y)), max(abs_bits(v.z), abs_bits(v.w)));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_mov(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}

// Maximum over aligned groups of WIDTH lanes (2 .. 64), left in every lane of
// the group.  Quad permutations give the maximum of each 4 lanes; mirroring
// each half row (lane i <-> 7 - i) then each row (i <-> 15 - i) pairs every
// 4- then 8-lane group with its neighbour; v_permlane16_swap exchanges rows
// 0 <-> 1 and 2 <-> 3, v_permlane32_swap the two halves of the wave.
template <int WIDTH>
__device__ __forceinline__ uint32_t group_max_bits(uint32_t v) {
  static_assert(WIDTH >= 2 && WIDTH <= 64 && (WIDTH & (WIDTH - 1)) == 0, "group width");
  v = max(v, dpp_mov<0xB1>(v));  // quad_perm [1, 0, 3, 2]
  if constexpr (WIDTH >= 4) v = max(v, dpp_mov<0x4E>(v));   // quad_perm [2, 3, 0, 1]
  if constexpr (WIDTH >= 8) v = max(v, dpp_mov<0x141>(v));  // row_half_mirror
  if constexpr (WIDTH >= 16) v = max(v, dpp_mov<0x140>(v));  // row_mirror
  if constexpr (WIDTH >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(uint32_t(p[0]), uint32_t(p[1]));
  }
  if constexpr (WIDTH >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(uint32_t(p[0]), uint32_t(p[1]));
  }
  return v;
}

// Four float32 in [-fmax, fmax] to four fp8 codes (first value in the low
// byte), nearest with ties to even.
__device__ __forceinline__ uint32_t cvt4_e4m3(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}
__device__ __forceinline__ uint32_t cvt4_e5m2(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_bf8_f32(c, d, lo, true));
}

// ------------------------------------------------------------ MX (e8m0) --
// Exponent of the block scale: the smallest E with max(amax, 1e-10) <=
// fmax * 2^E, read off the float32 fields.  fmax = 1.75 * 2^EMAX for both
// formats (448 = 1.75 * 2^8, 57344 = 1.75 * 2^15).
template <int EMAX>
__device__ __forceinline__ int mx_exponent(float amax) {
  const uint32_t u = __float_as_uint(fmaxf(amax, scale_floor()));
  const int e = int((u >> 23) & 0xFFu) - 127;
  const int E = e - EMAX + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(E, -127), 127);
}

// x * 2^-E (exact) clamped to the format's range, four at a time.
template <int CODE>  // 0 = e4m3, 1 = e5m2
__device__ __forceinline__ uint32_t mx_encode4(const float* x, int E) {
  constexpr float fmax = CODE == 0 ? kE4M3Max : kE5M2Max;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __builtin_amdgcn_fmed3f(ldexpf(x[i], -E), -fmax, fmax);
  return CODE == 0 ? cvt4_e4m3(y[0], y[1], y[2], y[3]) : cvt4_e5m2(y[0], y[1], y[2], y[3]);
}

// Loads 8 consecutive source values as float (from f32 or bf16).
template <int SRC_BF16>
__device__ __forceinline__ void load8(const void* base, int64_t elem, float (&x)[8]) {
  if (SRC_BF16) {
    const uint4 w = ldnt(
        reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem));
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = decode_bf16(p[i] & 0xFFFFu);
      x[2 * i + 1] = decode_bf16(p[i] >> 16);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    const float4 a = ldnt(f);
    const float4 b = ldnt(f + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// Stores 8 consecutive values (as f32, or as bf16 rounded to nearest even).
template <int BF16>
__device__ __forceinline__ void store8(void* p, int64_t elem, const float (&v)[8]) {
  if (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = encode_bf16(v[2 * i]) | (encode_bf16(v[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + elem) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + elem);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace bsq
