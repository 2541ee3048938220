// Layer and rms norm, whose output may leave as the next product's operand,
// and their gradients.
//
//   mean = sum x / C (rms: 0), rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),
//   xn = (x - mean) rstd, y = xn gamma + beta
//   d = dy gamma, dx = rstd (d - xn (sum d xn) / C - (sum d) / C), the last
//   term for layer norm only; dgamma = sum over rows of dy xn, dbeta of dy
//
// in float32.  The variance is summed from x - mean in a second pass over the
// registers, so that rows far from zero do not cancel.  Where a sum or a square
// passes float32, or squares are too small for it, the row is taken again times
// the power of two that brings its largest value below 1.  Codes are of the
// float32 y, before y's own rounding.
//
// Bound by memory where a row has enough values to fill its threads.  A row stays
// in the registers of NT threads, P times eight values each; rows too long for
// that are read again instead.  The weights'
// gradients are summed by groups of rows in registers, a group's sums go to the
// workspace, and a second kernel adds the groups in their order, so that every
// run gives the same bytes.
#include "fp4.h"
#include "moe_index.h"
#include "norm.h"

#include <type_traits>

namespace bsq {

namespace {

// Sum over a wave, left in each lane, by exchanges between registers (through
// LDS, as shuffles, each of the six takes five times as long).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp_mov<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v = dpp_add<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v = dpp_add<0x141>(v);  // row_half_mirror
  v = dpp_add<0x140>(v);  // row_mirror
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
// Sum over NT threads (64: a wave of its own), left in each; `red` is one of
// two or more places used in turn.
template <int NT>
__device__ __forceinline__ float sum_over(float v, float* red) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[i];
  }
  return v;
}
template <int NT>
__device__ __forceinline__ void sum_over(float& a, float& b, float* red) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    const int w = int(threadIdx.x >> 6) % W;
    if ((threadIdx.x & 63) == 0) {
      red[w] = a;
      red[W + w] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += red[i];
      b += red[W + i];
    }
  }
}

constexpr uint32_t kInfinity = 0x7F800000u;
// Whether float32 held the sums of a row, by its variance and eps (the same in
// every lane): they are finite, and the squares (each off by 2^-150 at most) are
// not lost beside them.  500000 x 128 bfloat16 rms 118 us, 114 without the check;
// from 512 columns on the same.
__device__ __forceinline__ bool held(float v) {
  constexpr uint32_t kLeast = 0x0D800000u;  // 2^-100
  return __builtin_expect(uint32_t(__builtin_amdgcn_readfirstlane(int(__float_as_uint(v)))) - kLeast < kInfinity - kLeast, 1);
}
// The power of two k for a row that it did not hold: the largest magnitude (its
// bits are `top`) times 2^-k is below 1, and so is eps times 2^-2k; 2^-k is a
// float32.
__device__ __forceinline__ int exponent_of(uint32_t top, float eps) {
  const float m = fmaxf(__uint_as_float(top), eps < __builtin_inff() ? sqrtf(eps) : 0.f);
  return max(m > 0.f ? __builtin_amdgcn_frexp_expf(m) : 0, -126);
}
// 1 / sqrt of such a row's variance and eps, both times 2^-2k.  A row of one
// value has zeros to normalise, beside which eps counts however small it is: it
// goes on as it was.
__device__ __forceinline__ float rstd_again(float var, float eps, float& mean, int& k) {
  if (var == 0.f) {
    mean = ldexpf(mean, k);
    k = 0;
  }
  return 1.0f / sqrtf(var + ldexpf(eps, -2 * k));
}
// Largest of magnitudes' bits over NT threads, left in each.
template <int NT>
__device__ __forceinline__ uint32_t max_over(uint32_t v, float* red) {
  v = group_max_bits<64>(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
    v = 0u;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v = max(v, __float_as_uint(red[i]));
  }
  return v;
}

template <int BF16>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  return BF16 ? decode_bf16(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}
template <int BF16>
__device__ __forceinline__ void store1(void* p, int64_t at, float v) {
  if (BF16) static_cast<uint16_t*>(p)[at] = uint16_t(bf16_pair(v, v) & 0xFFFFu);
  else static_cast<float*>(p)[at] = v;
}

// The columns that a thread of a row's NT holds: VEC eight neighbours P times,
// else 8 P single ones NT apart.
template <int NT, int VEC>
__device__ __forceinline__ int col(int t, int p, int i) {
  return VEC ? 8 * (t + NT * p) + i : t + NT * (8 * p + i);
}
template <int BF16, int NT, int VEC>
__device__ __forceinline__ void load_row(const void* base, int64_t row0, int t, int p, int C, float (&v)[8]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (8 * (t + NT * p) < C) load8<BF16>(base, row0 + 8 * (t + NT * p), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col<NT, 0>(t, p, i) < C ? load1<BF16>(base, row0 + col<NT, 0>(t, p, i)) : 0.f;
  }
}
// Eight values as they lie in memory, so that a row under way takes as few
// registers as it can.
template <int BF16, int NT, int VEC>
struct Raw {
  uint4 v[BF16 && VEC ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t row0, int t, int p, int C) {
    if constexpr (VEC) {
      v[0] = make_uint4(0u, 0u, 0u, 0u);
      if (!BF16) v[1] = v[0];
      const int64_t at = row0 + 8 * (t + NT * p);
      if (8 * (t + NT * p) < C) {
        if constexpr (BF16) {
          v[0] = ldnt(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
        } else {
          v[0] = ldnt(reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at));
          v[1] = ldnt(reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at) + 1);
        }
      }
    } else {
      float x[8];
      load_row<BF16, NT, 0>(base, row0, t, p, C, x);
      v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (BF16 && VEC) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = decode_bf16(w[i] & 0xFFFFu);
        x[2 * i + 1] = decode_bf16(w[i] >> 16);
      }
    } else {
      const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
};
template <int BF16, int NT, int VEC>
__device__ __forceinline__ void store_row(void* base, int64_t row0, int t, int p, int C, const float (&v)[8]) {
  if constexpr (VEC) {
    if (8 * (t + NT * p) < C) store8<BF16>(base, row0 + 8 * (t + NT * p), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col<NT, 0>(t, p, i) < C) store1<BF16>(base, row0 + col<NT, 0>(t, p, i), v[i]);
  }
}
// gamma or beta of the thread's columns; `none` where it is null.
template <int NT, int VEC>
__device__ __forceinline__ void load_weight(const float* w, int t, int p, int C, float none, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = none;
  if (w == nullptr) return;
  if constexpr (VEC) {
    if (8 * (t + NT * p) < C) {
      const float4* f = reinterpret_cast<const float4*>(w + 8 * (t + NT * p));
      const float4 a = f[0], b = f[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col<NT, 0>(t, p, i) < C) v[i] = w[col<NT, 0>(t, p, i)];
  }
}

// Eight neighbours of a row as codes, four lanes to a block; every lane of the
// wave takes part, `in` guards the stores.
__device__ __forceinline__ void put_codes(NormCode code, uint8_t* codes, uint8_t* scales, int64_t at, bool in,
                                          bool words, const float (&v)[8]) {
  if (code == NormCode::e2m1) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    const uint32_t e = mx4_byte(group_max_bits<4>(m));
    put_scale4<4>(scales, at / 32, in, words, e);
    if (in) *reinterpret_cast<uint32_t*>(codes + at / 2) = encode8_fp4(v, mx_scale(e));
  } else if (code == NormCode::e4m3) {
    put_row<0>(codes, scales, at / 8, in, words, v);
  } else {
    put_row<1>(codes, scales, at / 8, in, words, v);
  }
}

// ---------------------------------------------------------------- forward --
// Workgroups go through the rows blockIdx.x + gridDim.x i (of kRows rows each),
// gamma and beta in registers, the next one's load under way.  16384 x 4096
// bfloat16 to bfloat16 and e4m3 58-69 us, 5.0-5.8 TB/s (a copy reaches 5.1), to
// bfloat16 and e2m1 50, to e2m1 alone 45; one row 2.7 us.  Rows that leave lanes
// idle are bound by their instructions: 524288 x 128 155 us, 1.7 TB/s, 262144 x 64
// 70 us, 1.0.
template <int BF16, int VEC, int NT, int P>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_norm(NormLaunch a) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;  // of a workgroup
  __shared__ float red[2][2][NT > 64 ? NT / 64 : 1], again[3][NT > 64 ? NT / 64 : 1];
  const int t = threadIdx.x % NT, sub = threadIdx.x / NT, C = int(a.C);
  const int64_t step = int64_t(gridDim.x) * kRows;
  saturate_fp8();
  Raw<BF16, NT, VEC> raw[P];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int p = 0; p < P; ++p) raw[p].load(a.x, (r < a.R ? r : a.R - 1) * a.C, t, p, C);
  };
  load(int64_t(blockIdx.x) * kRows + sub);
  float g[P][8], b[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    load_weight<NT, VEC>(a.gamma, t, p, C, 1.f, g[p]);
    load_weight<NT, VEC>(a.beta, t, p, C, 0.f, b[p]);
  }
  const bool words = VEC && C % 128 == 0 && aligned4(a.scales);
  int buf = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < a.R; r0 += step, buf ^= 1) {
    const int64_t r = r0 + sub, row0 = r * a.C;
    const bool in = r < a.R;
    float x[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) raw[p].get(x[p]);
    if (r0 + step < a.R) load(r + step);
    float mean = 0.f, s = 0.f;
    if (!a.rms) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[p][i];
      mean = sum_over<NT>(s, red[buf][0]) / float(C);
      s = 0.f;
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[p][i] = col<NT, VEC>(t, p, i) < C ? x[p][i] - mean : 0.f;
        s += x[p][i] * x[p][i];
      }
    const float var = sum_over<NT>(s, red[buf][1]) / float(C);
    float rstd = 1.0f / sqrtf(var + a.eps);
    int k = 0;
    if (!held(var + a.eps)) {  // all threads of the row; x is read again, and y not yet written
      uint32_t top = 0u;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        load_row<BF16, NT, VEC>(a.x, (in ? r : a.R - 1) * a.C, t, p, C, x[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, abs_bits(x[p][i]));
      }
      top = max_over<NT>(top, again[0]);
      rstd = __builtin_nanf("");  // an infinity or NaN makes the whole row NaN
      if (top < kInfinity) {
        k = exponent_of(top, a.eps);
        mean = s = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < 8; ++i) s += x[p][i] = ldexpf(x[p][i], -k);
        // no further out than the row's values, so that 2^k times it is finite
        const float most = ldexpf(__uint_as_float(top), -k);
        if (!a.rms) mean = __builtin_amdgcn_fmed3f(sum_over<NT>(s, again[1]) / float(C), -most, most);
        s = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[p][i] = col<NT, VEC>(t, p, i) < C ? x[p][i] - mean : 0.f;
            s += x[p][i] * x[p][i];
          }
        rstd = rstd_again(sum_over<NT>(s, again[2]) / float(C), a.eps, mean, k);
      }
    }
    if (t == 0 && in) {
      if (a.mean != nullptr) a.mean[r] = ldexpf(mean, k);
      if (a.rstd != nullptr) a.rstd[r] = ldexpf(rstd, -k);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[p][i] = x[p][i] * rstd * g[p][i] + b[p][i];
      if (in && a.y != nullptr) store_row<BF16, NT, VEC>(a.y, row0, t, p, C, x[p]);
      if (VEC && a.codes != nullptr)
        put_codes(a.code, a.codes, a.scales, row0 + 8 * (t + NT * p), in && 8 * (t + NT * p) < C, words, x[p]);
    }
  }
}

// Any length: a workgroup reads its row three times.  A thread's share of a sum
// is long, so the mean is summed from the row's first value on, and mended by
// that of x - mean, which the second pass brings: rows far from zero are as good
// as others at any length, and a row of one value is zeros.
constexpr int kLong = 1024;
template <int BF16>
__global__ void __launch_bounds__(kLong) k_norm_long(NormLaunch a, int64_t first) {
  __shared__ float red[3][kLong / 64], pairs[2][2 * kLong / 64];
  const int64_t r = first + blockIdx.x, row0 = r * a.C;
  saturate_fp8();
  // `again`: the row is taken times 2^-k
  constexpr std::false_type no{};
  constexpr std::true_type yes{};
  int k = 0;
  float down = 1.f;
  auto at = [&](int64_t c, auto again) {
    const float x = load1<BF16>(a.x, row0 + c);
    return decltype(again)::value ? x * down : x;
  };
  float mean = 0.f;
  auto variance = [&](float* red_mean, float* red_var, auto again) {
    float s = 0.f, left = 0.f;
    if (a.rms) {
      for (int64_t c = threadIdx.x; c < a.C; c += kLong) s += at(c, again) * at(c, again);
      return sum_over<kLong>(s, red_var) / float(a.C);
    }
    const float x0 = at(0, again);
    for (int64_t c = threadIdx.x; c < a.C; c += kLong) s += at(c, again) - x0;
    mean = x0 + sum_over<kLong>(s, red_mean) / float(a.C);
    s = 0.f;
    for (int64_t c = threadIdx.x; c < a.C; c += kLong) {
      const float d = at(c, again) - mean;
      left += d;
      s += d * d;
    }
    sum_over<kLong>(s, left, red_var);
    left /= float(a.C);
    mean += left;
    const float v = s / float(a.C) - left * left;
    return v < 0.f ? 0.f : v;
  };
  const float var = variance(red[0], pairs[0], no);
  float rstd = 1.0f / sqrtf(var + a.eps);
  if (!held(var + a.eps)) {
    uint32_t top = 0u;
    for (int64_t c = threadIdx.x; c < a.C; c += kLong) top = max(top, abs_bits(at(c, no)));
    top = max_over<kLong>(top, red[1]);
    rstd = __builtin_nanf("");  // an infinity or NaN makes the whole row NaN
    if (top < kInfinity) {
      k = exponent_of(top, a.eps);
      down = ldexpf(1.f, -k);
      const float scaled = variance(red[2], pairs[1], yes), most = __uint_as_float(top) * down;
      mean = __builtin_amdgcn_fmed3f(mean, -most, most);  // so that 2^k times it is finite
      rstd = rstd_again(scaled, a.eps, mean, k);
    }
  }
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[r] = ldexpf(mean, k);
    if (a.rstd != nullptr) a.rstd[r] = ldexpf(rstd, -k);
  }
  auto write = [&](auto again) {
    auto value = [&](int64_t c) {
      const float xn = (at(c, again) - mean) * rstd;
      return xn * (a.gamma != nullptr ? a.gamma[c] : 1.f) + (a.beta != nullptr ? a.beta[c] : 0.f);
    };
    if (a.codes == nullptr) {
      if (a.y == nullptr) return;
      for (int64_t c = threadIdx.x; c < a.C; c += kLong) store1<BF16>(a.y, row0 + c, value(c));
      return;
    }
    // blocks of 32, four lanes of eight neighbours each; a wave's lanes go on
    // together, since the maximum of a block is taken across them
    for (int64_t c0 = 0; c0 < a.C; c0 += 8 * kLong) {
      const int64_t c = c0 + 8 * threadIdx.x;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c < a.C ? value(c + i) : 0.f;
      if (c < a.C && a.y != nullptr) store8<BF16>(a.y, row0 + c, v);
      put_codes(a.code, a.codes, a.scales, row0 + c, c < a.C, false, v);
    }
  };
  if (k == 0) write(no);
  else write(yes);
}

// --------------------------------------------------------------- backward --
// (x - mean) rstd, of halves where the row is so large that the difference may
// pass float32.
struct Centre {
  float h, mean, rstd;
  __device__ __forceinline__ Centre(float m, float r)
      : h(r < 0x1p-64f ? 0.5f : 1.0f), mean(m * h), rstd(r < 0x1p-64f ? r + r : r) {}
  __device__ __forceinline__ float operator()(float x) const { return fmaf(x, h, -mean) * rstd; }
};

// Workgroups go through the rows blockIdx.x + gridDim.x i (of kRows rows each),
// the next one's loads under way while a row is summed and written.  Two rows
// of 256 threads to a workgroup halve the groups' sums: 16384 x 4096 71 + 5 us
// against 73 + 7, 5.9 TB/s.  Rows of 8193 and more have 1024 threads, whose 128
// registers do not hold two rows under way, gamma and both sums: some are spilled
// in the loop (11 of bfloat16, 82 of float32, 97 of single values), 4096 x 16384
// bfloat16 116 us, 3.5 TB/s, float32 331 us, 2.4.
template <int NT>
constexpr int rows_of = NT < 256 ? 256 / NT : NT == 256 ? 2 : 1;
template <int BF16, int VEC, int NT, int P>
__global__ void __launch_bounds__(NT * rows_of<NT>) k_norm_dx(NormBackwardLaunch a) {
  constexpr int kRows = rows_of<NT>;
  __shared__ float reds[kRows][2][2 * (NT > 64 ? NT / 64 : 1)];
  __shared__ float join[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? 2 * 8 * P * NT : 1];
  const int t = threadIdx.x % NT, sub = threadIdx.x / NT, C = int(a.C);
  float(*const red)[2 * (NT > 64 ? NT / 64 : 1)] = reds[sub];
  const float inv = 1.0f / float(C);
  const int64_t step = int64_t(gridDim.x) * kRows;
  Raw<BF16, NT, VEC> xr[P], dr[P];
  float mean_r = 0.f, rstd_r = 0.f;
  auto load = [&](int64_t r) {
    const int64_t rr = r < a.R ? r : a.R - 1;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      xr[p].load(a.x, rr * a.C, t, p, C);
      dr[p].load(a.dy, rr * a.C, t, p, C);
    }
    mean_r = a.rms ? 0.f : a.mean[rr];
    rstd_r = a.rstd[rr];
  };
  load(int64_t(blockIdx.x) * kRows + sub);
  float g[P][8], sg[P][8], sb[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    load_weight<NT, VEC>(a.gamma, t, p, C, 1.f, g[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[p][i] = sb[p][i] = 0.f;
  }
  int buf = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < a.R; r0 += step, buf ^= 1) {
    const int64_t r = r0 + sub;
    const bool in = r < a.R;
    float x[P][8], dy[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      xr[p].get(x[p]);
      dr[p].get(dy[p]);
    }
    const Centre norm(mean_r, rstd_r);
    const float rstd = rstd_r;
    if (r0 + step < a.R) load(r + step);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // columns and rows that are not there have dy 0
        const float d = in ? dy[p][i] : 0.f, xn = in ? norm(x[p][i]) : 0.f;
        x[p][i] = xn;
        sg[p][i] += d * xn;
        sb[p][i] += d;
        dy[p][i] = d * g[p][i];
        s1 += dy[p][i] * (col<NT, VEC>(t, p, i) < C ? xn : 0.f);
        s2 += dy[p][i];
      }
    sum_over<NT>(s1, s2, red[buf]);
    s1 *= inv;
    s2 = a.rms ? 0.f : s2 * inv;
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[p][i] = rstd * (dy[p][i] - x[p][i] * s1 - s2);
      if (in) store_row<BF16, NT, VEC>(a.dx, r * a.C, t, p, C, x[p]);
    }
  }
  if (a.dgamma == nullptr && a.dbeta == nullptr) return;
  if constexpr (kRows > 1) {  // the rows of the workgroup, in their order
    if (sub > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          join[sub - 1][(8 * p + i) * NT + t] = sg[p][i];
          join[sub - 1][(8 * (P + p) + i) * NT + t] = sb[p][i];
        }
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int o = 0; o < kRows - 1; ++o)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sg[p][i] += join[o][(8 * p + i) * NT + t];
          sb[p][i] += join[o][(8 * (P + p) + i) * NT + t];
        }
  }
  float* const to = a.space + int64_t(blockIdx.x) * C;
  float* const to_b = to + int64_t(gridDim.x) * C;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    store_row<0, NT, VEC>(to, 0, t, p, C, sg[p]);
    store_row<0, NT, VEC>(to_b, 0, t, p, C, sb[p]);
  }
}

// Any length: a row's sums, then its gradient, from two reads.
template <int BF16>
__global__ void __launch_bounds__(kLong) k_norm_dx_long(NormBackwardLaunch a, int64_t first) {
  __shared__ float red[2 * kLong / 64];
  const int64_t r = first + blockIdx.x, row0 = r * a.C;
  const float rstd = a.rstd[r];
  const Centre norm(a.rms ? 0.f : a.mean[r], rstd);
  float s1 = 0.f, s2 = 0.f;
  for (int64_t c = threadIdx.x; c < a.C; c += kLong) {
    const float d = load1<BF16>(a.dy, row0 + c) * (a.gamma != nullptr ? a.gamma[c] : 1.f);
    s1 += d * norm(load1<BF16>(a.x, row0 + c));
    s2 += d;
  }
  sum_over<kLong>(s1, s2, red);
  s1 /= float(a.C);
  s2 = a.rms ? 0.f : s2 / float(a.C);
  for (int64_t c = threadIdx.x; c < a.C; c += kLong) {
    const float d = load1<BF16>(a.dy, row0 + c) * (a.gamma != nullptr ? a.gamma[c] : 1.f);
    const float xn = norm(load1<BF16>(a.x, row0 + c));
    store1<BF16>(a.dx, row0 + c, rstd * (d - xn * s1 - s2));
  }
}
// The weights' gradients of long rows: a thread to a column, groups of rows.
template <int BF16>
__global__ void __launch_bounds__(256) k_norm_dw_long(NormBackwardLaunch a, int groups) {
  const int64_t chunks = up_to(a.C, 256), c = (int64_t(blockIdx.x) % chunks) * 256 + threadIdx.x;
  const int64_t gr = int64_t(blockIdx.x) / chunks;
  if (c >= a.C) return;
  float sg = 0.f, sb = 0.f;
  for (int64_t r = gr; r < a.R; r += groups) {
    const float d = load1<BF16>(a.dy, r * a.C + c);
    sg += d * Centre(a.rms ? 0.f : a.mean[r], a.rstd[r])(load1<BF16>(a.x, r * a.C + c));
    sb += d;
  }
  a.space[gr * a.C + c] = sg;
  a.space[(groups + gr) * a.C + c] = sb;
}

// Sums over the groups: 16 columns x 16 shares of the groups, each in their
// order, the shares added through LDS.
constexpr int kSumCols = 16, kShares = 16;
__global__ void __launch_bounds__(kSumCols* kShares) k_norm_sum(const float* __restrict__ space, int groups, int64_t C,
                                                                float* dgamma, float* dbeta) {
  __shared__ float part[kShares][kSumCols];
  const int64_t chunks = up_to(C, kSumCols);
  const int which = int(blockIdx.x / chunks);  // 0: dgamma, 1: dbeta
  float* const out = which ? dbeta : dgamma;
  if (out == nullptr) return;
  const int x = threadIdx.x % kSumCols, share = threadIdx.x / kSumCols;
  const int64_t c = blockIdx.x % chunks * kSumCols + x;
  const int per = (groups + kShares - 1) / kShares, end = min(groups, (share + 1) * per);
  float s = 0.f;
  if (c < C) {
#pragma unroll 16
    for (int i = share * per; i < end; ++i) s += space[(int64_t(which) * groups + i) * C + c];
  }
  part[share][x] = s;
  __syncthreads();
  if (share > 0 || c >= C) return;
#pragma unroll
  for (int i = 1; i < kShares; ++i) s += part[i][x];
  out[c] = s;
}

// Threads of a row and how many times eight values each holds: f(NT, P).
template <typename F>
bsq_status with_shape(int64_t C, F&& f) {
#define BSQ_NORM(NT, P) f(std::integral_constant<int, NT>{}, std::integral_constant<int, P>{})
  if (C <= 512) return BSQ_NORM(64, 1);
  if (C <= 1024) return BSQ_NORM(64, 2);
  if (C <= 2048) return BSQ_NORM(256, 1);
  if (C <= 4096) return BSQ_NORM(256, 2);
  if (C <= 8192) return BSQ_NORM(512, 2);
  return BSQ_NORM(1024, 2);
#undef BSQ_NORM
}
constexpr int64_t kInRegisters = 16384;

}  // namespace

bsq_status launch_norm(const NormLaunch& L, hipStream_t st) {
  if (L.C > kInRegisters)
    return in_parts(L.R, kLaunchGroups / 2, [&](int64_t first, int64_t n) {
      if (L.bf16) hipLaunchKernelGGL((k_norm_long<1>), dim3(unsigned(n)), kLong, 0, st, L, first);
      else hipLaunchKernelGGL((k_norm_long<0>), dim3(unsigned(n)), kLong, 0, st, L, first);
      return launch_status("norm");
    });
  return with_shape(L.C, [&](auto nt, auto p) {
    constexpr int NT = decltype(nt)::value, P = decltype(p)::value, kRows = NT < 256 ? 256 / NT : 1;
    // eight workgroups of 256 threads to a CU
    const int64_t most = 8 * kCUs * 256 / (NT < 256 ? 256 : NT), all = up_to(L.R, kRows);
    const dim3 g = dim3(unsigned(all < most ? all : most)), b = dim3(NT < 256 ? 256 : NT);
    switch ((L.bf16 ? 1 : 0) | (L.C % 8 == 0 ? 2 : 0)) {
      case 0: hipLaunchKernelGGL((k_norm<0, 0, NT, P>), g, b, 0, st, L); break;
      case 1: hipLaunchKernelGGL((k_norm<1, 0, NT, P>), g, b, 0, st, L); break;
      case 2: hipLaunchKernelGGL((k_norm<0, 1, NT, P>), g, b, 0, st, L); break;
      default: hipLaunchKernelGGL((k_norm<1, 1, NT, P>), g, b, 0, st, L);
    }
    return launch_status("norm");
  });
}

bsq_status launch_norm_backward(const NormBackwardLaunch& L, hipStream_t st) {
  const bool weights = L.dgamma != nullptr || L.dbeta != nullptr;
  int groups = 0;
  bsq_status s = BSQ_OK;
  if (L.R > 0 && L.C > kInRegisters) {
    if (weights) {  // first: dx may take the place of x or dy
      groups = int(L.R < 32 ? L.R : 32);
      const dim3 g = dim3(unsigned(up_to(L.C, 256) * groups));
      if (L.bf16) hipLaunchKernelGGL((k_norm_dw_long<1>), g, 256, 0, st, L, groups);
      else hipLaunchKernelGGL((k_norm_dw_long<0>), g, 256, 0, st, L, groups);
      s = launch_status("norm_backward (weights)");
      if (s != BSQ_OK) return s;
    }
    s = in_parts(L.R, kLaunchGroups / 2, [&](int64_t first, int64_t n) {
      if (L.bf16) hipLaunchKernelGGL((k_norm_dx_long<1>), dim3(unsigned(n)), kLong, 0, st, L, first);
      else hipLaunchKernelGGL((k_norm_dx_long<0>), dim3(unsigned(n)), kLong, 0, st, L, first);
      return launch_status("norm_backward");
    });
  } else if (L.R > 0) {
    s = with_shape(L.C, [&](auto nt, auto p) {
      constexpr int NT = decltype(nt)::value, P = decltype(p)::value, kRows = rows_of<NT>;
      const int64_t most = NT == 256 ? 256 : 512, all = up_to(L.R, kRows);
      groups = int(all < most ? all : most);
      const dim3 g = dim3(unsigned(groups)), b = dim3(NT * kRows);
      switch ((L.bf16 ? 1 : 0) | (L.C % 8 == 0 ? 2 : 0)) {
        case 0: hipLaunchKernelGGL((k_norm_dx<0, 0, NT, P>), g, b, 0, st, L); break;
        case 1: hipLaunchKernelGGL((k_norm_dx<1, 0, NT, P>), g, b, 0, st, L); break;
        case 2: hipLaunchKernelGGL((k_norm_dx<0, 1, NT, P>), g, b, 0, st, L); break;
        default: hipLaunchKernelGGL((k_norm_dx<1, 1, NT, P>), g, b, 0, st, L);
      }
      return launch_status("norm_backward");
    });
  }
  if (s != BSQ_OK || !weights) return s;
  hipLaunchKernelGGL(k_norm_sum, dim3(unsigned(2 * up_to(L.C, kSumCols))), kSumCols * kShares, 0, st, L.space, groups, L.C, L.dgamma, L.dbeta);
  return launch_status("norm_backward (weights)");
}

}  // namespace bsq
