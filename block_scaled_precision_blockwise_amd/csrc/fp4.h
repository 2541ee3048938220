// Device helpers of the kernels that write e2m1 codes (magnitudes 0, 0.5, 1,
// 1.5, 2, 3, 4, 6; two to a byte, the lower index in the low nibble).
#pragma once

#include "fp8.h"

namespace bsq {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// E8M0 byte of a block from the bits of its largest magnitude: E + 127 for the
// least E with max(amax, 1e-10) <= 6 * 2^E.  6 = 1.5 * 2^2, so a significand
// above 1.5 carries into the exponent.  NaN gives the NaN scale; infinity the
// byte of the largest finite magnitudes.
__device__ __forceinline__ uint32_t mx4_byte(uint32_t bits) {
  const uint32_t e = ((max(bits, __float_as_uint(scale_floor())) + 0x3FFFFFu) >> 23) - 2u;
  return bits > 0x7F800000u ? 0xFFu : e;
}

// Eight values times 2^-E as codes, nearest even; `scale` is 2^E.  The
// conversion saturates at 6.
__device__ __forceinline__ uint32_t encode8_fp4(const float (&x)[8], float scale) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0], x[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2], x[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6], x[7], scale, 3);
}
__device__ __forceinline__ uint32_t encode8_fp4(const uint32_t (&x)[4], float scale) {  // of bfloat16 pairs
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, x[0]), scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, x[1]), scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, x[2]), scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, x[3]), scale, 3);
}

// nvfp4: E4M3 byte of a block's scale, max(amax / 6, 2^-9) rounded to nearest
// even and at most 448, from the bits of its largest magnitude.  NaN gives NaN.
__device__ __forceinline__ uint32_t nv4_byte(uint32_t bits) {
  const float s = __builtin_amdgcn_fmed3f(__uint_as_float(bits) / 6.0f, 0.001953125f, 448.0f);
  const uint32_t q = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(s, s, 0, false)) & 0xFFu;
  return bits > 0x7F800000u ? 0x7Fu : q;
}
__device__ __forceinline__ float nv4_scale(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8(int(byte), 0); }

// The scale of a block of SPAN lanes, `at` its place.  Where the four blocks of
// 4 SPAN lanes are all there and start a word, one lane writes the word.
template <int SPAN>
__device__ __forceinline__ void put_scale4(uint8_t* scales, int64_t at, bool in, bool words, uint32_t e) {
  const int lane = int(threadIdx.x & 63u);
  if (words) {
    uint32_t w = e | (lane_ahead<SPAN>(e) << 8);
    w |= lane_ahead<2 * SPAN>(w) << 16;
    if (in && lane % (4 * SPAN) == 0) *reinterpret_cast<uint32_t*>(scales + at) = w;
  } else if (in && lane % SPAN == 0) {
    scales[at] = uint8_t(e);
  }
}

}  // namespace bsq
