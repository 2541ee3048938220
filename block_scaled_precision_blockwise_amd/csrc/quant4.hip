// Quantizer to e2m1 codes, along rows and / or transposed from one read.
//
//   mxfp4  blocks of 32: E the least integer with max(amax, 1e-10) <= 6 2^E,
//          codes of x 2^-E
//   nvfp4  blocks of 16, y = x f: s = e4m3(min(max(amax / 6, 2^-9), 448)),
//          codes of y / s, a true division
//
// both rounded to nearest even.  For mxfp4 one instruction scales and rounds a
// pair.  The quotient of nvfp4 is rounded to float32 first, which moves no
// code: the borders between codes times s have 8 significant bits, and a y
// beside one differs from it by more than half a step of the quotient.
#include "fp4.h"
#include "moe_index.h"
#include "quant4.h"

namespace bsq {

namespace {

// Eight neighbours of a row, SPAN lanes to a block: its codes, and the scale byte.
template <int NV, int SPAN>
__device__ __forceinline__ uint32_t code8(const float (&x)[8], uint32_t& byte) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
  m = group_max_bits<SPAN>(m);
  if constexpr (NV) {
    byte = nv4_byte(m);
    const float s = nv4_scale(byte);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] / s;
    return encode8_fp4(y, 1.0f);
  } else {
    byte = mx4_byte(m);
    return encode8_fp4(x, mx_scale(byte));
  }
}

// ------------------------------------------------------------------- rows --
// A stream of blocks, eight values per thread, U of them under way.  mxfp4 is
// bound by memory: 8 x 4096 x 4096 bfloat16 54 us, 6.3 TB/s, float32 110 us, 5.5;
// one row of 4096 2.0.  nvfp4 is bound by its divisions: the same bfloat16 values
// 82 us, 4133 x 1072 float32 7.8; with products by one reciprocal of the scale,
// which round otherwise, 55 and 6.5.
template <int BF16, int NV>
__global__ void __launch_bounds__(256) k_fp4_rows(const void* __restrict__ src, const float* __restrict__ factor,
                                                  uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                  int64_t n8, int64_t first) {
  constexpr int U = 4, SPAN = NV ? 2 : 4;
  const float f = NV && factor != nullptr ? *factor : 1.0f;
  const bool words = aligned4(scales);
  const int64_t base = (first + blockIdx.x) * (256 * U) + threadIdx.x;
  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
    if (base + 256 * u < n8) load8<BF16>(src, (base + 256 * u) * 8, x[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = base + 256 * u;
    const bool in = at < n8;
    if (NV) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] *= f;
    }
    uint32_t e;
    const uint32_t q = code8<NV, SPAN>(x[u], e);
    if (in) codes[at] = q;
    // a word of scales that the array ends in goes by bytes
    const bool whole = (at | int64_t(4 * SPAN - 1)) < n8;
    put_scale4<SPAN>(scales, at / SPAN, in && whole, words, e);
    if (in && !whole && threadIdx.x % SPAN == 0) scales[at / SPAN] = uint8_t(e);
  }
}

// ------------------------------------------------------------------ tiles --
// 128 x 128 values go through LDS, so that one read gives both ways round.
// bfloat16 values stay pairs of two rows (32 KiB), float32 ones are floats.
// Eight lanes own a column, 16 rows each.  mxfp4 is bound by memory: 8 x 4096 x
// 4096 bfloat16 values both ways round, 411 MB in 87 us, 4.7 TB/s (a copy reaches
// 5.1); nvfp4 by two divisions a value, 183 us (99 with a block's reciprocal).
// The transposed codes' stores are non-temporal, the rows' are not: 99 us
// without, 101 with both (a row's 64 bytes of a tile are half a line, which the
// L2 joins with its neighbour's).
struct Tile4Args {
  const void* src;
  const float* factor;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t R, C, first;
  int tiles_r, tiles_c;
};

template <int BF16, int NV>
__global__ void __launch_bounds__(256) k_fp4_tile(Tile4Args a, int64_t total) {
  constexpr int kBlock = NV ? 16 : 32, SPAN = NV ? 2 : 4, SPANT = NV ? 1 : 2;
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTile * kTile / (BF16 ? 2 : 1)];
  const float f = NV && a.factor != nullptr ? *a.factor : 1.0f;
  const int64_t t = xcd_run(a.first + blockIdx.x, total), per = int64_t(a.tiles_r) * a.tiles_c;
  const int64_t b = t / per, in_b = t - b * per;
  const int64_t r0 = in_b / a.tiles_c * kTile, c0 = in_b % a.tiles_c * kTile;
  const int64_t base = b * a.R * a.C;
  const int tx = threadIdx.x, c8 = tx & 15;
  const int64_t c = c0 + 8 * c8;

  const bool words = a.C % kTile == 0 && aligned4(a.scales);
  auto put = [&](int64_t r, const float (&x)[8]) {
    const bool in = r < a.R && c < a.C;
    uint32_t e;
    const uint32_t q = code8<NV, SPAN>(x, e);
    const int64_t at = base + r * a.C + c;
    if (in) *reinterpret_cast<uint32_t*>(a.codes + at / 2) = q;
    put_scale4<SPAN>(a.scales, at / kBlock, in, words, e);
  };
  auto put_pairs = [&](int64_t r, const uint32_t (&x)[4]) {  // of bfloat16, mxfp4
    const bool in = r < a.R && c < a.C;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_u16x2(m, x[i] & 0x7FFF7FFFu);
    const uint32_t e = mx4_byte(group_max_bits<4>(max(m & 0xFFFFu, m >> 16)) << 16);
    const int64_t at = base + r * a.C + c;
    if (in) *reinterpret_cast<uint32_t*>(a.codes + at / 2) = encode8_fp4(x, mx_scale(e));
    put_scale4<4>(a.scales, at / 32, in, words, e);
  };
  if constexpr (BF16) {
    const uint16_t* x = static_cast<const uint16_t*>(a.src) + base;
    uint4 v[4][2];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t r = r0 + 2 * ((tx >> 4) + 16 * s) + h;
        v[s][h] = make_uint4(0u, 0u, 0u, 0u);
        if (r < a.R && c < a.C) v[s][h] = ldnt(reinterpret_cast<const uint4*>(x + r * a.C + c));
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int rp = (tx >> 4) + 16 * s;
      const uint32_t lo[4] = {v[s][0].x, v[s][0].y, v[s][0].z, v[s][0].w};
      const uint32_t hi[4] = {v[s][1].x, v[s][1].y, v[s][1].z, v[s][1].w};
      if (!NV && a.codes != nullptr) {
        put_pairs(r0 + 2 * rp, lo);
        put_pairs(r0 + 2 * rp + 1, hi);
      } else if (a.codes != nullptr) {
        float y[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t* p = h ? hi : lo;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[2 * i] = decode_bf16(p[i] & 0xFFFFu) * f;
            y[2 * i + 1] = decode_bf16(p[i] >> 16) * f;
          }
          put(r0 + 2 * rp + h, y);
        }
      }
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
  } else {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int rr = (tx >> 4) + 16 * s;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (r0 + rr < a.R && c < a.C) load8<0>(a.src, base + (r0 + rr) * a.C + c, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= f;
      if (a.codes != nullptr) put(r0 + rr, x);
      float4* o = reinterpret_cast<float4*>(tile + tile_at<0>(rr, c8));
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
  __syncthreads();

  const int share = tx & 7;
  const int64_t r = r0 + 16 * share;
  const bool words_t = a.R % kTile == 0 && aligned4(a.scales_t);
#pragma unroll
  for (int it = 0; it < kTile * 8 / 256; ++it) {
    const int oc = (tx >> 3) + 32 * it;
    const int64_t co = c0 + oc;
    const bool in = r < a.R && co < a.C;
    uint32_t e, q[2];
    if constexpr (BF16 && !NV) {
      uint32_t x[2][4], m = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i / 4][i & 3] = tile[tile_at<1>(8 * share + i, oc >> 3) + (oc & 7)];
        m = max_u16x2(m, x[i / 4][i & 3] & 0x7FFF7FFFu);
      }
      e = mx4_byte(group_max_bits<2>(max(m & 0xFFFFu, m >> 16)) << 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) q[h] = encode8_fp4(x[h], mx_scale(e));
    } else {
      float x[2][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (BF16) {
          const uint32_t w = tile[tile_at<1>(8 * share + i, oc >> 3) + (oc & 7)];
          x[i / 4][2 * (i & 3)] = decode_bf16(w & 0xFFFFu) * f;
          x[i / 4][2 * (i & 3) + 1] = decode_bf16(w >> 16) * f;
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x[h][i] = __uint_as_float(tile[tile_at<0>(16 * share + 8 * h + i, oc >> 3) + (oc & 7)]);
        }
      }
      uint32_t m = 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[h][i]));
      if constexpr (NV) {
        e = nv4_byte(m);
        const float s = nv4_scale(e);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[h][i] = x[h][i] / s;
          q[h] = encode8_fp4(x[h], 1.0f);
        }
      } else {
        e = mx4_byte(group_max_bits<2>(m));
#pragma unroll
        for (int h = 0; h < 2; ++h) q[h] = encode8_fp4(x[h], mx_scale(e));
      }
    }
    const int64_t at = base + co * a.R + r;
    put_scale4<SPANT>(a.scales_t, at / kBlock, in, words_t, e);
    if (in) stnt(a.codes_t + at / 2, q[0], q[1]);
  }
}

}  // namespace

bsq_status launch_quant4(const Quant4Launch& L, hipStream_t st) {
  if (L.codes_t == nullptr) {
    const int64_t n8 = L.B * L.R * L.C / 8;
    return in_parts(up_to(n8, 1024), kLaunchGroups, [&](int64_t first, int64_t n) {
      const dim3 g = dim3(unsigned(n));
      uint32_t* codes = reinterpret_cast<uint32_t*>(L.codes);
      switch ((L.bf16 ? 1 : 0) | (L.nv ? 2 : 0)) {
        case 0: hipLaunchKernelGGL((k_fp4_rows<0, 0>), g, 256, 0, st, L.src, L.factor, codes, L.scales, n8, first); break;
        case 1: hipLaunchKernelGGL((k_fp4_rows<1, 0>), g, 256, 0, st, L.src, L.factor, codes, L.scales, n8, first); break;
        case 2: hipLaunchKernelGGL((k_fp4_rows<0, 1>), g, 256, 0, st, L.src, L.factor, codes, L.scales, n8, first); break;
        default: hipLaunchKernelGGL((k_fp4_rows<1, 1>), g, 256, 0, st, L.src, L.factor, codes, L.scales, n8, first);
      }
      return launch_status("quant_fp4");
    });
  }
  Tile4Args a{L.src, L.factor, L.codes, L.scales, L.codes_t, L.scales_t, L.R, L.C, 0, int(up_to(L.R, kTile)),
              int(up_to(L.C, kTile))};
  const int64_t total = L.B * a.tiles_r * a.tiles_c;
  return in_parts(total, kLaunchGroups, [&](int64_t first, int64_t n) {
    const dim3 g = dim3(unsigned(n));
    a.first = first;
    switch ((L.bf16 ? 1 : 0) | (L.nv ? 2 : 0)) {
      case 0: hipLaunchKernelGGL((k_fp4_tile<0, 0>), g, 256, 0, st, a, total); break;
      case 1: hipLaunchKernelGGL((k_fp4_tile<1, 0>), g, 256, 0, st, a, total); break;
      case 2: hipLaunchKernelGGL((k_fp4_tile<0, 1>), g, 256, 0, st, a, total); break;
      default: hipLaunchKernelGGL((k_fp4_tile<1, 1>), g, 256, 0, st, a, total);
    }
    return launch_status("quant_fp4 (both ways round)");
  });
}

}  // namespace bsq
