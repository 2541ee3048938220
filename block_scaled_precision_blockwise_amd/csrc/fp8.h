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

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two values as bfloat16, to nearest even; NaN of any payload stays NaN
// (encode_bf16 carries some of them into the sign).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Stores 8 consecutive values (as f32, or as bf16 rounded to nearest even).
template <int BF16>
__device__ __forceinline__ void store8(void* p, int64_t elem, const float (&v)[8]) {
  if (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + elem) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + elem);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// ------------------------------------- tiles written in both orientations --
// A workgroup of NT threads holds a 128 x 128 tile in LDS and writes its
// codes transposed: eight lanes own a column, 16 rows (16 bytes) each, so
// that one store instruction writes whole 128-byte lines; two neighbouring
// lanes share a block of 32 rows.  Chunks of eight columns are XORed with the
// lane's share of the rows, so that the 64 lanes' reads (8 columns x 8
// shares) fall on 64 banks and the writers keep 16-byte stores.
constexpr int kTile = 128;

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

__device__ __forceinline__ bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The conversions below saturate (MODE.FP16_OVFL), so that an infinite value
// takes the largest code, as the clamp of mx_encode4 gives it.
__device__ __forceinline__ void saturate_fp8() { __builtin_amdgcn_s_setreg(1 | (23 << 6), 1); }

// Four values times 2^-E as codes; `scale` is 2^E.  Two at a time in one
// instruction, which rounds once, to nearest even.
template <int CODE>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float scale) {
  s16x2 q{};
  if constexpr (CODE == 0) {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, a, b, scale, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, c, d, scale, true);
  } else {
    q = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(q, a, b, scale, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(q, c, d, scale, true);
  }
  return __builtin_bit_cast(uint32_t, q);
}
template <int CODE>
__device__ __forceinline__ uint32_t encode4(uint32_t ab, uint32_t cd, float scale) {  // of bfloat16 pairs
  const bf16x2 x = __builtin_bit_cast(bf16x2, ab), y = __builtin_bit_cast(bf16x2, cd);
  s16x2 q{};
  if constexpr (CODE == 0) {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, x, scale, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, y, scale, true);
  } else {
    q = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(q, x, scale, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(q, y, scale, true);
  }
  return __builtin_bit_cast(uint32_t, q);
}
// mx_exponent plus 127 from the bits of a block's largest magnitude: the scale
// byte, and 23 places up the scale 2^E itself.  The significand passes 1.75
// where adding 2^23 - 1 - 0x600000 carries into the exponent; from the floor
// on no clamp can be reached.
template <int CODE>
__device__ __forceinline__ uint32_t mx_byte(uint32_t bits) {
  return ((max(bits, __float_as_uint(scale_floor())) + 0x1FFFFFu) >> 23) - (CODE == 0 ? 8u : 15u);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Stores that nothing reads again soon: they leave the L2 to what is shared.
__device__ __forceinline__ void stnt(void* p, uint32_t a, uint32_t b) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(u32x2_t{a, b}, static_cast<u32x2_t*>(p));
}
__device__ __forceinline__ void stnt(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  __builtin_nontemporal_store(u32x4_t{a, b, c, d}, static_cast<u32x4_t*>(p));
}

// store8 as such a store.
template <int BF16>
__device__ __forceinline__ void store8nt(void* p, int64_t elem, const float (&v)[8]) {
  if (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    stnt(static_cast<uint16_t*>(p) + elem, u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      stnt(static_cast<float*>(p) + elem + 4 * i, __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
           __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  }
}

// Values of the lane N further on in the row of 16 (its first 16 - N lanes).
template <int N>
__device__ __forceinline__ uint32_t lane_ahead(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x100 + N, 0xF, 0xF, true));
}

// The scale of block f8 / 4 of a row of 16 lanes, four lanes to a block.  Where
// the row's four blocks are all there and start a word, one lane writes the
// word: a byte at a time cost 15 of 133 us.
__device__ __forceinline__ void put_scale(uint8_t* scales, int64_t f8, bool in, bool words, uint32_t e) {
  if (words) {
    uint32_t w = e | (lane_ahead<4>(e) << 8);
    w |= lane_ahead<8>(w) << 16;
    if (in && (threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(scales + (f8 >> 2)) = w;
  } else if (in && (f8 & 3) == 0) {
    scales[f8 >> 2] = uint8_t(e);
  }
}

// Eight neighbours of a row, four lanes to a block, 16 to the tile's row:
// codes and scale (`words`: see put_scale).  The
// values are floats, or four words of bfloat16 pairs.  Every lane of the wave
// takes part in the maximum; `in` guards the stores.
template <int CODE>
__device__ __forceinline__ void put_row(uint8_t* codes, uint8_t* scales, int64_t f8, bool in, bool words,
                                        const float (&x)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
  const uint32_t E = mx_byte<CODE>(group_max_bits<4>(m));
  const float s = mx_scale(E);
  put_scale(scales, f8, in, words, E);
  if (in) stnt(codes + 8 * f8, encode4<CODE>(x[0], x[1], x[2], x[3], s), encode4<CODE>(x[4], x[5], x[6], x[7], s));
}
template <int CODE>
__device__ __forceinline__ void put_row(uint8_t* codes, uint8_t* scales, int64_t f8, bool in, bool words,
                                        const uint32_t (&x)[4]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_u16x2(m, x[i] & 0x7FFF7FFFu);
  m = group_max_bits<4>(max(m & 0xFFFFu, m >> 16));
  const uint32_t E = mx_byte<CODE>(m << 16);
  const float s = mx_scale(E);
  put_scale(scales, f8, in, words, E);
  if (in) stnt(codes + 8 * f8, encode4<CODE>(x[0], x[1], s), encode4<CODE>(x[2], x[3], s));
}

// Where tile keeps eight columns from 8 c8 of row `r` (a float each), or of
// the pair of rows `r` (one word, the even row in the low half).
template <int PAIRS>
__device__ __forceinline__ int tile_at(int r, int c8) {
  return r * kTile + 8 * (c8 ^ ((r >> (PAIRS ? 3 : 4)) & 7));
}

// The tile at rows r0 .., columns c0 .. as codes_t [cols, rows].
template <int CODE, int PAIRS, int NT>
__device__ __forceinline__ void put_columns(const uint32_t* tile, int64_t r0, int64_t c0, int64_t rows, int64_t cols,
                                            uint8_t* codes_t, uint8_t* scales_t) {
  const int share = threadIdx.x & 7;
  const int64_t r = r0 + 16 * share;
  const bool words = rows % kTile == 0 && aligned4(scales_t);
#pragma unroll
  for (int it = 0; it < kTile * 8 / NT; ++it) {
    const int oc = (threadIdx.x >> 3) + NT / 8 * it;
    const int64_t c = c0 + oc;
    const bool in = r < rows && c < cols;
    uint32_t q[4], E;
    if constexpr (PAIRS) {
      uint32_t x[8], m = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = tile[tile_at<1>(8 * share + i, oc >> 3) + (oc & 7)];
        m = max_u16x2(m, x[i] & 0x7FFF7FFFu);
      }
      E = mx_byte<CODE>(group_max_bits<2>(max(m & 0xFFFFu, m >> 16)) << 16);
      const float s = mx_scale(E);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = encode4<CODE>(x[2 * i], x[2 * i + 1], s);
    } else {
      float x[16];
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] = __uint_as_float(tile[tile_at<0>(16 * share + i, oc >> 3) + (oc & 7)]);
        m = max(m, abs_bits(x[i]));
      }
      E = mx_byte<CODE>(group_max_bits<2>(m));
      const float s = mx_scale(E);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = encode4<CODE>(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], s);
    }
    if (words) {
      uint32_t w = E | (lane_ahead<2>(E) << 8);
      w |= lane_ahead<4>(w) << 16;
      if (in && share == 0) *reinterpret_cast<uint32_t*>(scales_t + c * (rows / 32) + r / 32) = w;
    } else if (in && (share & 1) == 0) {
      scales_t[c * (rows / 32) + r / 32] = uint8_t(E);
    }
    if (in) stnt(codes_t + c * rows + r, q[0], q[1], q[2], q[3]);
  }
}

// Tile number of workgroup L of n: workgroups are dealt to the 8 XCDs
// round-robin, and XCD x takes the x-th contiguous eighth of the tiles.
__device__ __forceinline__ int64_t xcd_run(int64_t L, int64_t n) {
  const int64_t per = n / 8;
  return L < 8 * per ? (L & 7) * per + (L >> 3) : L;
}

}  // namespace bsq
