// Routing to experts and its gradient.
//
//   p = softmax(x) or 1 / (1 + e^-x) over a token's E logits,
//   c = p + bias, and a group of experts is worth the sum of its group_top
//   largest c; the k largest c of the top_groups best groups are chosen (the
//   lowest index of equals), with weights p (over their sum, where
//   renormalised) times scale.
//
// The choice is a discrete answer: it is made on scores in 64 bits, so that
// two experts whose scores differ only past the 24th bit are still put in
// their true order.
//
// Bound by instruction issue: 32768 tokens of 256 experts (sigmoid, bias, 4 of
// 8 groups, 8 choices, all scores) take 32 us for 50 MB (137 us with a token
// to a wave and rounds of argmax, 40 with the exponential's coefficients moved
// into registers before each use and branches around each score); its
// gradient 17 us for 67 MB (23 us with a token to a wave and 2-byte loads).
// One token: 4.2 us, 12 before.
#include <math.h>

#include <type_traits>

#include "fp8.h"
#include "moe.h"
#include "moe_index.h"

namespace bsq {

namespace {

struct RouteArgs {
  int64_t T;
  int E, k, groups, top_groups, group_top;
  const void* logits;
  int sigmoid, renorm;
  float scale;
  const float* bias;
  int32_t* ids;
  float* weights;
  float* scores;
};

template <int BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  return BF16 ? decode_bf16(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Values o .. o + 3 of a row of n; `none` past its end.  `whole`: rows are
// whole fours, aligned.
template <int BF16>
__device__ __forceinline__ void load4(const void* base, int64_t row, int o, int n, bool whole, float none, float* x) {
  if (whole) {
    if (o >= n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = none;
    } else if (BF16) {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + row + o);
      x[0] = decode_bf16(v.x & 0xFFFFu);
      x[1] = decode_bf16(v.x >> 16);
      x[2] = decode_bf16(v.y & 0xFFFFu);
      x[3] = decode_bf16(v.y >> 16);
    } else {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row + o);
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = o + i < n ? logit_at<BF16>(base, row + o + i) : none;
  }
}

// Over a row of 16 lanes, left in each.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp_mov<0xB1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_mov<0x4E>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_mov<0x141>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(dpp_mov<0x140>(__float_as_uint(v))));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp_mov<0xB1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<0x4E>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<0x141>(__float_as_uint(v)));
  return v + __uint_as_float(dpp_mov<0x140>(__float_as_uint(v)));
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = fmax(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// A choice's share of the sum of p over the choices, before the division: e^(x
// - m), or e^-m / (1 + e^-x), m the largest chosen x, of sigmoids at most 0.
// p itself is nothing where a bias has steered the choice to logits that lie
// 750 below the row's largest; the share is not.
__device__ __forceinline__ double share(bool sigmoid, double x, double m) {
  if (x == -INFINITY) return 0.0;
  if (!sigmoid) return exp(x - m);
  return exp(fmin(x, 0.0) - fmin(m, 0.0)) / (1.0 + exp(-fabs(x)));
}

// One token by one wave, in 64 bits: lane l holds logits l, l + 64, ...
// `cs` is E doubles of LDS that belong to this wave.
template <int BF16, int EPL>
__device__ void route_token(const RouteArgs& a, int64_t t, int lane, double* cs) {
  const int E = a.E;
  double p[EPL], c[EPL];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    p[i] = e < E ? double(logit_at<BF16>(a.logits, t * E + e)) : -INFINITY;
    top = fmax(top, p[i]);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = 1.0 / (1.0 + exp(-p[i]));
  } else {
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // a row of -inf alone has scores of zero
      p[i] = p[i] == -INFINITY ? 0.0 : exp(p[i] - top);
      sum += p[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = sum == 0.0 ? 0.0 : p[i] / sum;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    c[i] = p[i];
    if (e < E) {
      if (a.bias != nullptr) c[i] += double(a.bias[e]);
      if (a.scores != nullptr) a.scores[t * E + e] = float(p[i]);
    }
    if (!(c[i] == c[i])) c[i] = -INFINITY;  // NaN: chosen last, so that every id is one of the experts
  }
  if (a.groups > 1) {
    const int per = E / a.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 64 * i < E) cs[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double worth = -INFINITY;
    if (lane < a.groups) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < per; ++j) {
        const double v = cs[lane * per + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      worth = a.group_top == 2 ? b1 + b2 : b1;
    }
    int before = 0;  // groups that come before this lane's
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(worth, g);
      before += (o > worth || (o == worth && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / per)) & 1)) c[i] = -INFINITY;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // k rounds: the best of what is left, the lowest index of equals
  uint32_t taken = 0u;
  double w_mine = 0.0;
  int id_mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY, pb = 0.0;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((taken >> i) & 1u) && (at == 0x7FFFFFFF || c[i] > best)) {
        best = c[i];
        pb = p[i];
        at = e;
      }
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
      const double ob = __shfl_xor(best, m), op = __shfl_xor(pb, m);
      const int oa = __shfl_xor(at, m);
      if (oa != 0x7FFFFFFF && (at == 0x7FFFFFFF || ob > best || (ob == best && oa < at))) {
        best = ob;
        pb = op;
        at = oa;
      }
    }
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
    if (lane == j) {
      id_mine = at;
      w_mine = pb;
    }
  }
  if (a.renorm) {
    const double x = lane < a.k ? double(logit_at<BF16>(a.logits, t * E + id_mine)) : -INFINITY;
    const double s = share(a.sigmoid, x, wave_max(x)), total = wave_sum(s);
    // a row with NaN or +inf has softmax scores of NaN, also where none of them is chosen
    w_mine = w_mine == w_mine ? (total == 0.0 ? 0.0 : s / total) : w_mine;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id_mine;
    a.weights[t * a.k + lane] = float(w_mine * double(a.scale));
  }
}

template <int BF16, int EPL>
__global__ void __launch_bounds__(256) k_route(RouteArgs a) {
  __shared__ double cs[4][64 * EPL];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t t = int64_t(blockIdx.x) * 4 + w; t < a.T; t += int64_t(gridDim.x) * 4)
    route_token<BF16, EPL>(a, t, lane, cs[w]);
}

// ------------------------------------------------- few choices, fast path --
// A token by L lanes (16: four tokens to a wave; 64), each with S scores.
// The choice is a sort instead of rounds of argmax: a score's low 10 bits
// make room for its expert's number, so that one 64-bit maximum orders scores
// and breaks ties by the lowest index; every lane sorts its keys and keeps
// 8, and log2(L) exchanges merge the lists (the larger of A[i] and B[7 - i]
// are the 8 largest of two sorted lists).  Scores that are closer than the
// lost bits and this path's own exponential allow are told apart by the general
// path above, unless their logits and biases are the same.  A score is off by
// at most 2^-40.5 of itself (the exponential's 2^-41.5, and as much by the sum),
// a key by 2^-42 more of its value c, so the difference of two by less than
// (p + p' + |c|) 2^-40; what lies within (p + p' + |c|) 2^-38 is settled there,
// and groups within (|worth| + 2) 2^-38, four scores of at most 1 each.
constexpr int kTop = 8;

// e^x to a relative 2^-41.5 for x <= 0 or so: x = n ln 2 + r (ln 2 in two
// pieces, the first of 36 bits, so that n times it is exact), the power series of
// e^r to r^10 (|r| <= ln 2 / 2: what it leaves out is below 2.2e-13, at r = -ln 2
// / 2 1.31 2^-42 of e^r).
struct ExpSeries {
  double c[8];  // 1 / 10!, ..., 1 / 3!
  __device__ ExpSeries()
      : c{1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0} {
    // kept in registers: as constants they would be moved there before each use
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("" : "+v"(c[i]));
  }
  __device__ __forceinline__ double operator()(double x) const {
    x = __builtin_fmax(x, -800.0);  // 2^-1154: zero either way
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = fma(n, -0x1.62e42fefa0000p-1, x);
    r = fma(n, -0x1.cf79abc9e3b3ap-40, r);
    double y = c[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) y = fma(y, r, c[i]);
    y = fma(y, r, 0.5);
    y = fma(y, r, 1.0);
    y = fma(y, r, 1.0);
    return __builtin_ldexp(y, int(n));
  }
};

// 1 / d for 1 <= d < 2^1000: the hardware's start and one Newton step.
__device__ __forceinline__ double recip_near(double d) {
  const double y = __builtin_amdgcn_rcp(d);
  return fma(y, fma(-d, y, 1.0), y);
}

constexpr double kFar = 690.0;
__device__ __forceinline__ double sigmoid_near(const ExpSeries& exp_near, double x) {
  // 0 from e^690 on (kFar), where the true score is below 2^-995
  const double p = recip_near(1.0 + exp_near(__builtin_fmin(-x, kFar)));
  return x < -kFar ? 0.0 : p;
}

union Bits64 {
  double d;
  int64_t i;
  uint32_t u[2];
};

// The value of the lane that step STEP pairs with this one (STEP 0 .. 3:
// within rows of 16).
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  // quad permutations, then the half row and the row mirrored: every lane has a source
  constexpr int kCtrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), kCtrl, 0xF, 0xF, true));
}
// Both values of the pair, in an order that both lanes agree on or not (for
// commutative use); steps 4 and 5 exchange rows and halves.
template <int STEP>
__device__ __forceinline__ void pair(double v, double& a, double& b) {
  Bits64 x{v}, p, q;
  if constexpr (STEP < 4) {
    p.u[0] = partner<STEP>(x.u[0]);
    p.u[1] = partner<STEP>(x.u[1]);
    a = v;
    b = p.d;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto s = STEP == 4 ? __builtin_amdgcn_permlane16_swap(x.u[h], x.u[h], false, false)
                               : __builtin_amdgcn_permlane32_swap(x.u[h], x.u[h], false, false);
      p.u[h] = uint32_t(s[0]);
      q.u[h] = uint32_t(s[1]);
    }
    a = p.d;
    b = q.d;
  }
}

template <int N, typename F>
__device__ __forceinline__ void steps(F&& f) {
  if constexpr (N > 0) {
    steps<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}
template <int L>
constexpr int kLog = L == 16 ? 4 : 6;

template <int L>
__device__ __forceinline__ double lanes_max(double v) {
  steps<kLog<L>>([&](auto s) {
    double a, b;
    pair<decltype(s)::value>(v, a, b);
    v = __builtin_fmax(a, b);
  });
  return v;
}
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
  steps<kLog<L>>([&](auto s) {
    double a, b;
    pair<decltype(s)::value>(v, a, b);
    v = a + b;
  });
  return v;
}

__device__ __forceinline__ void order2(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi;
  b = lo;
}
// Descending order of 8 (19 exchanges).
__device__ __forceinline__ void sort8(double* v) {
  order2(v[0], v[2]); order2(v[1], v[3]); order2(v[4], v[6]); order2(v[5], v[7]);
  order2(v[0], v[4]); order2(v[1], v[5]); order2(v[2], v[6]); order2(v[3], v[7]);
  order2(v[0], v[1]); order2(v[2], v[3]); order2(v[4], v[5]); order2(v[6], v[7]);
  order2(v[2], v[4]); order2(v[3], v[5]);
  order2(v[1], v[4]); order2(v[3], v[6]);
  order2(v[1], v[2]); order2(v[3], v[4]); order2(v[5], v[6]);
}
// Descending order of 8 that rise and fall once.
__device__ __forceinline__ void merge8(double* v) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order2(v[i], v[i + d]);
}

constexpr double kNever = -1.7e308;  // key of an expert that has no score to be chosen by
// Below kTiny a key has no room for the expert's number beside what orders it
// (and sigmoid_near is 0 for scores that are not): such choices are settled by
// the general path if a logit is kFar to 760 below (from 746 on scores are 0 in
// 64 bits).  Below kSmall the chosen scores' sum is no divisor for what may be
// left of a score.
constexpr double kTiny = 1e-290, kSmall = 1e-250;

// The general path as a call, so that its registers are not this path's.
template <int BF16, int EPL>
__device__ __attribute__((noinline)) void route_token_apart(RouteArgs a, int64_t t, int lane, double* cs) {
  route_token<BF16, EPL>(a, t, lane, cs);
}

template <int BF16, int SIGMOID, int L, int S>
__global__ void __launch_bounds__(256) k_route_top(RouteArgs a) {
  const ExpSeries exp_near;
  constexpr int kSlow = L * S / 64;  // scores per lane of the general path
  __shared__ double cs[4][64 * kSlow];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int E = a.E, G = a.groups, per = E / G;
  const int LG = L / G, shift = 31 - __clz(LG);    // lanes per group
  const int l = lane & (L - 1), g = l >> shift, lg = l & (LG - 1);
  constexpr int V = 4;                            // neighbours in a lane
  const bool whole = (per & (V - 1)) == 0;        // rows and groups start at whole fours
  constexpr int TPW = 64 / L;
  const int64_t t0 = (int64_t(blockIdx.x) * 4 + w) * TPW;
  if (t0 >= a.T) return;
  const int64_t t_mine = t0 + lane / L;
  const bool live = t_mine < a.T;
  const int64_t row = (live ? t_mine : a.T - 1) * E;

  // slot i is expert (in its group) of chunk i / 4
  auto at = [&](int i) { return (i / V * LG + lg) * V + (i & (V - 1)); };
  float x[S];
#pragma unroll
  for (int q = 0; q < S / V; ++q)
    load4<BF16>(a.logits, row + g * per, at(q * V), per, whole, -INFINITY, x + 4 * q);
  float largest = x[0];  // NaN if there is one
#pragma unroll
  for (int i = 1; i < S; ++i) largest = __builtin_elementwise_maximum(largest, x[i]);
  // ---- scores
  double c[S];
  double top = 0.0, inv = 0.0;
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < S; ++i) c[i] = sigmoid_near(exp_near, double(x[i]));
  } else {
    top = lanes_max<L>(double(largest));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      // a row of -inf alone has scores of zero
      const double v = exp_near(double(x[i]) - top);
      c[i] = x[i] == -INFINITY ? 0.0 : v;
      sum += c[i];
    }
    sum = lanes_sum<L>(sum);
    inv = sum == 0.0 ? 0.0 : recip_near(sum);
#pragma unroll
    for (int i = 0; i < S; ++i) c[i] *= inv;
  }
  if (a.scores != nullptr && live) {
#pragma unroll
    for (int q = 0; q < S / V; ++q) {
      const int o = at(q * V);
      float* p = a.scores + row + g * per + o;
      if (whole) {
        if (o < per)
          *reinterpret_cast<float4*>(p) =
              make_float4(float(c[4 * q]), float(c[4 * q + 1]), float(c[4 * q + 2]), float(c[4 * q + 3]));
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (o + i < per) p[i] = float(c[4 * q + i]);
      }
    }
  }
  // ---- what the choice goes by
  if (a.bias != nullptr) {
#pragma unroll
    for (int q = 0; q < S / V; ++q) {
      float b[V];
      load4<0>(a.bias, g * per, at(q * V), per, whole, 0.f, b);
#pragma unroll
      for (int i = 0; i < V; ++i) c[V * q + i] += double(b[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int o = at(i);
    // infinities stay numbers beside the expert's number; NaN comes last
    c[i] = __builtin_fmin(__builtin_fmax(c[i], kNever), -kNever);
    if (o >= per) c[i] = -INFINITY;
  }
  bool in = true, tiny = false;
  // for the general path to settle, which shows NaN where it is
  bool close = SIGMOID ? largest != largest : !(largest < INFINITY);
  if (G > 1) {
    double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      b2 = __builtin_fmax(b2, __builtin_fmin(b1, c[i]));
      b1 = __builtin_fmax(b1, c[i]);
    }
    steps<kLog<L>>([&](auto s) {
      if ((1 << decltype(s)::value) < LG) {
        double a1, o1, a2, o2;
        pair<decltype(s)::value>(b1, a1, o1);
        pair<decltype(s)::value>(b2, a2, o2);
        b1 = __builtin_fmax(a1, o1);
        b2 = __builtin_fmax(__builtin_fmin(a1, o1), __builtin_fmax(a2, o2));
      }
    });
    const double worth = a.group_top == 2 ? b1 + b2 : b1;
    tiny = fabs(worth) < kTiny;
    int before = 0;  // groups that come before this lane's
    for (int h = 1; h < G; ++h) {
      const int og = (g + h) & (G - 1);
      const double o = __shfl(worth, (lane & ~(L - 1)) + (og << shift));
      before += (o > worth || (o == worth && og < g)) ? 1 : 0;
      close |= o != worth && fabs(o - worth) <= (fabs(worth) + 2.0) * 0x1p-38;
    }
    in = before < a.top_groups;
  }
  double list[S > kTop ? S : kTop];
  double key[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    Bits64 b{in || c[i] == -INFINITY ? c[i] : kNever};
    const uint32_t e = uint32_t(g * per + at(i));
    if (c[i] != -INFINITY) b.u[0] = (b.u[0] & ~1023u) | (b.i < 0 ? e : 1023u - e);
    key[i] = list[i] = b.d;
  }
#pragma unroll
  for (int i = S; i < kTop; ++i) list[i] = -INFINITY;
  sort8(list);
  if constexpr (S > kTop) {
    sort8(list + kTop);
#pragma unroll
    for (int i = 0; i < kTop; ++i) list[i] = __builtin_fmax(list[i], list[2 * kTop - 1 - i]);
    merge8(list);
  }
  steps<kLog<L>>([&](auto s) {
    double p[kTop], q[kTop];
#pragma unroll
    for (int i = 0; i < kTop; ++i) pair<decltype(s)::value>(list[i], p[i], q[i]);
#pragma unroll
    for (int i = 0; i < kTop; ++i) list[i] = __builtin_fmax(p[i], q[kTop - 1 - i]);
    merge8(list);
  });
  // ---- lane j has the j-th choice
  Bits64 mine{list[0]};
  double last = list[0];
#pragma unroll
  for (int j = 1; j < kTop; ++j) {
    if (l == j) mine.d = list[j];
    if (a.k - 1 == j) last = list[j];
  }
  const bool on = l < a.k;
  int id = int(mine.u[0] & 1023u);
  if (mine.i >= 0) id = 1023 - id;
  id = id < E ? id : E - 1;
  const float xm = logit_at<BF16>(a.logits, row + id);
  const double bm = a.bias != nullptr ? double(a.bias[id]) : 0.0;
  double p = 0.0;
  if (on) p = SIGMOID ? sigmoid_near(exp_near, double(xm)) : xm == -INFINITY ? 0.0 : exp_near(double(xm) - top) * inv;
  const double total = lanes_sum<16>(p);

  // ---- neighbours in the order, and the last against what was left out
  const double next = __shfl_down(mine.d, 1), p_next = __shfl_down(p, 1), b_next = __shfl_down(bm, 1);
  const float x_next = __shfl_down(xm, 1);
  close |= l + 1 < a.k && next > kNever * 0.999 &&
               fabs(mine.d - next) <= (fabs(mine.d) + p + p_next) * 0x1p-38 && !(xm == x_next && bm == b_next);
  close |= a.renorm && on && xm != -INFINITY && total < kSmall;
  tiny |= on && fabs(mine.d) < kTiny;
  if (__ballot(tiny)) {
    const float from = SIGMOID ? 0.f : float(top);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float d = at(i) < per ? logit_at<BF16>(a.logits, row + g * per + at(i)) - from : 0.f;
      close |= d < float(-kFar) && d > -760.f;
    }
  }
  if (last > kNever * 0.999) {
    const int from = (lane & ~(L - 1)) + a.k - 1;
    const double lim = last - (fabs(last) + (a.bias != nullptr ? 1.0 : 0.0)) * 0x1p-38;
    bool more = false;
#pragma unroll
    for (int i = 0; i < S; ++i) more |= key[i] >= lim && key[i] < last;
    if (__ballot(more)) {
      const float xk = __shfl(xm, from);
      const double bk = __shfl(bm, from);
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (key[i] >= lim && key[i] < last) {
          const int e = g * per + at(i);
          close |= !(logit_at<BF16>(a.logits, row + e) == xk && (a.bias == nullptr || double(a.bias[e]) == bk));
        }
    }
  }
  const uint64_t again = __ballot(close && live);
  const uint64_t whose = L == 64 ? ~0ull : 0xFFFFull;
  if (on && live && !((again >> (lane & ~(L - 1))) & whose)) {
    a.ids[t_mine * a.k + l] = id;
    const double v = a.renorm ? (total == 0.0 ? 0.0 : p / total) : p;
    a.weights[t_mine * a.k + l] = float(v * double(a.scale));
  }
  if (again) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the scores above, which it writes anew
    for (int r = 0; r < TPW; ++r)
      if ((again >> (L * r)) & whose) route_token_apart<BF16, kSlow>(a, t0 + r, lane, cs[w]);
  }
}

// ------------------------------------------------------------- gradient --
struct RouteBwdArgs {
  int64_t T;
  int E, k;
  const void* logits;
  int sigmoid, renorm;
  float scale;
  const int32_t* ids;
  const float* dweights;
  const float* dscores;
  void* dlogits;
};

// Softmax dx = p (dp - sum p dp), sigmoid dx = dp p (1 - p), with dp the sum
// of dscores and, at a choice, of scale dw.  Renormalised, w = p / sum p over
// the choices: p dp is scale w (dw - sum w dw) there, and these sum to nothing
// over the choices.  w is an ordinary number also where p and the sum are
// nothing in 32 bits (a bias steers the choice only), so p dp is made of w, and
// w of e^x relative to the largest chosen x; 1 / sum p is never formed.

// A choice's share of the sum, before the division: e^(x - m), or e^-m /
// (1 + e^-x), m the largest chosen x, of sigmoids at most 0.
__device__ __forceinline__ float share(bool sigmoid, float x, float m) {
  if (x == -INFINITY) return 0.f;
  if (!sigmoid) return expf(x - m);
  const float r = 1.0f / (1.0f + expf(-fabsf(x)));
  return expf(fminf(x, 0.f) - fminf(m, 0.f)) * r;
}

// One wave per token; `dps` is E floats of LDS that belong to this wave.
template <int BF16, int EPL>
__device__ void route_backward_token(const RouteBwdArgs& a, int64_t t, int lane, float* dps) {
  const int E = a.E;
  float p[EPL], dp[EPL];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    p[i] = e < E ? logit_at<BF16>(a.logits, t * E + e) : -INFINITY;
    top = fmaxf(top, p[i]);
  }
  float q[EPL];  // 1 - p of the sigmoid, without the cancellation
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float z = expf(-fabsf(p[i])), r = 1.0f / (1.0f + z);
      q[i] = p[i] >= 0.f ? z * r : r;
      p[i] = p[i] >= 0.f ? r : z * r;
    }
  } else {
    top = wave_max(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = p[i] == -INFINITY ? 0.f : expf(p[i] - top);
      sum += p[i];
    }
    sum = wave_sum(sum);
    const float r = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= r;
  }
  const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
  const bool on = id >= 0 && id < E;
  const float xc = on ? logit_at<BF16>(a.logits, t * E + id) : -INFINITY;
  float d = on ? a.dweights[t * a.k + lane] * a.scale : 0.f;
  if (a.renorm) {
    const float s = share(a.sigmoid, xc, wave_max(xc)), total = wave_sum(s);
    const float w = total == 0.f ? 0.f : s / total;
    d = w * (d - wave_sum(w * d));
    if (a.sigmoid) d *= 1.0f / (1.0f + expf(xc));
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) dps[lane + 64 * i] = 0.f;
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  if (on) dps[id] = d;
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  float c[EPL], dot = 0.f;  // c: what the choices add to dx
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    c[i] = a.renorm ? dps[e] : 0.f;
    dp[i] = a.renorm ? 0.f : dps[e];
    if (a.dscores != nullptr && e < E) dp[i] += a.dscores[t * E + e];
    if (e < E) dot += p[i] * dp[i];
  }
  __builtin_amdgcn_wave_barrier();
  if (!a.sigmoid) dot = wave_sum(dot);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) {
      const float dx = c[i] + (a.sigmoid ? dp[i] * p[i] * q[i] : p[i] * (dp[i] - dot));
      if (BF16)
        static_cast<uint16_t*>(a.dlogits)[t * E + e] = uint16_t(bf16_pair(dx, 0.f));
      else
        static_cast<float*>(a.dlogits)[t * E + e] = dx;
    }
  }
}

template <int BF16, int EPL>
__global__ void __launch_bounds__(256) k_route_backward(RouteBwdArgs a) {
  __shared__ float dps[4][64 * EPL];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t t = int64_t(blockIdx.x) * 4 + w; t < a.T; t += int64_t(gridDim.x) * 4)
    route_backward_token<BF16, EPL>(a, t, lane, dps[w]);
}

// Four tokens to a wave, 16 lanes and 16 S experts each; lane l holds the
// choices l < k and the experts of chunks l, l + 16, ... of four.
template <int BF16, int S>
__global__ void __launch_bounds__(256) k_route_backward_rows(RouteBwdArgs a) {
  __shared__ __attribute__((aligned(16))) float dps[4][4][16 * S];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15;
  const int E = a.E;
  const int64_t t0 = (int64_t(blockIdx.x) * 4 + w) * 4;
  if (t0 >= a.T) return;
  const bool live = t0 + lane / 16 < a.T, whole = (E & 3) == 0;
  const int64_t t = live ? t0 + lane / 16 : a.T - 1, row = t * E;
  float* const mine = dps[w][lane / 16];
  // the chosen experts and their logits, while the row is on its way
  const int id = l < a.k ? a.ids[t * a.k + l] : -1;
  const bool on = id >= 0 && id < E;
  float d = on ? a.dweights[t * a.k + l] * a.scale : 0.f;
  const float xc = on ? logit_at<BF16>(a.logits, row + id) : -INFINITY;
  float p[S], ds[S];
#pragma unroll
  for (int q = 0; q < S / 4; ++q) {
    const int o = (q * 16 + l) * 4;
    load4<BF16>(a.logits, row, o, E, whole, -INFINITY, p + 4 * q);
    if (a.dscores != nullptr) load4<0>(a.dscores, row, o, E, whole, 0.f, ds + 4 * q);
    *reinterpret_cast<float4*>(mine + o) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __builtin_amdgcn_wave_barrier();
  if (!a.sigmoid) {
    float top = p[0];
#pragma unroll
    for (int i = 1; i < S; ++i) top = fmaxf(top, p[i]);
    top = row_max(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      p[i] = p[i] == -INFINITY ? 0.f : expf(p[i] - top);
      sum += p[i];
    }
    sum = row_sum(sum);
    const float r = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < S; ++i) p[i] *= r;
  }
  if (a.renorm) {
    const float s = share(a.sigmoid, xc, row_max(xc)), total = row_sum(s);
    const float w = total == 0.f ? 0.f : s / total;
    d = w * (d - row_sum(w * d));
    if (a.sigmoid) d *= 1.0f / (1.0f + expf(xc));
  }
  if (on) mine[id] = d;
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  float c[S], dp[S], dot = 0.f;  // c: what the choices add to dx
#pragma unroll
  for (int q = 0; q < S / 4; ++q) {
    const float4 v = *reinterpret_cast<const float4*>(mine + (q * 16 + l) * 4);
    const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[4 * q + i] = a.renorm ? u[i] : 0.f;
      dp[4 * q + i] = a.renorm ? 0.f : u[i];
    }
  }
  if (a.dscores != nullptr)
#pragma unroll
    for (int i = 0; i < S; ++i) dp[i] += ds[i];
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < S; ++i) dot = fmaf(p[i], dp[i], dot);
    dot = row_sum(dot);
  }
#pragma unroll
  for (int q = 0; q < S / 4; ++q) {
    float dx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * q + i;
      if (a.sigmoid) {
        // p and 1 - p, without the cancellation
        const float z = expf(-fabsf(p[j])), rz = 1.0f / (1.0f + z);
        dx[i] = c[j] + dp[j] * (z * rz) * rz;
      } else {
        dx[i] = c[j] + p[j] * (dp[j] - dot);
      }
    }
    const int o = (q * 16 + l) * 4;
    if (!live) continue;
    if (whole) {
      if (o < E) {
        if (BF16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + row + o) =
              make_uint2(bf16_pair(dx[0], dx[1]), bf16_pair(dx[2], dx[3]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + row + o) =
              make_float4(dx[0], dx[1], dx[2], dx[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (o + i < E) {
          if (BF16) static_cast<uint16_t*>(a.dlogits)[row + o + i] = uint16_t(bf16_pair(dx[i], 0.f));
          else static_cast<float*>(a.dlogits)[row + o + i] = dx[i];
        }
    }
  }
}

template <typename F>
void by_width(int E, F&& f) {
  const int epl = (E + 63) / 64;
  if (epl <= 1) f(std::integral_constant<int, 1>{});
  else if (epl <= 2) f(std::integral_constant<int, 2>{});
  else if (epl <= 4) f(std::integral_constant<int, 4>{});
  else if (epl <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

// From this many tokens on, four share a wave; below, a wave each fills more
// of the chip and is done sooner.  Forward, us of four to a wave against one:
// 1024 tokens of 256 experts 8.2 / 6.1, 2048 8.2 / 7.5, 4096 9.0 / 10.7; of
// 128 experts 5.3 / 5.2, 5.2 / 6.3, 5.6 / 9.3.
constexpr int64_t kRowTokens = 2048;

unsigned token_grid(int64_t T) {
  const int64_t g = (T + 3) / 4;
  return unsigned(g < 65536 ? g : 65536);
}

}  // namespace

static bsq_status route_part(const RouteLaunch& L, hipStream_t st) {
  const RouteArgs a{L.T, L.E, L.k, L.groups, L.top_groups, L.group_top, L.logits, L.sigmoid, L.renorm, L.scale,
                    L.bias, L.ids, L.weights, L.scores};
  const bool even = (L.groups & (L.groups - 1)) == 0;
  const int lanes = L.T >= kRowTokens && L.E <= 256 && L.groups <= 16 ? 16 : 64;
  if (even && L.k <= kTop) {
    const int slots = (L.E / L.groups + lanes / L.groups - 1) / (lanes / L.groups);
    if (slots <= 16) {
      const int64_t per = lanes == 16 ? 16 : 4, want = (L.T + per - 1) / per;
      const unsigned grid = unsigned(want);
      auto go = [&](auto l, auto s) {
        switch ((L.bf16 ? 1 : 0) | (L.sigmoid ? 2 : 0)) {
          case 0: hipLaunchKernelGGL((k_route_top<0, 0, l.value, s.value>), grid, 256, 0, st, a); break;
          case 1: hipLaunchKernelGGL((k_route_top<1, 0, l.value, s.value>), grid, 256, 0, st, a); break;
          case 2: hipLaunchKernelGGL((k_route_top<0, 1, l.value, s.value>), grid, 256, 0, st, a); break;
          default: hipLaunchKernelGGL((k_route_top<1, 1, l.value, s.value>), grid, 256, 0, st, a);
        }
      };
      auto by_slots = [&](auto l) {
        if (slots <= 4) go(l, std::integral_constant<int, 4>{});
        else if (slots <= 8) go(l, std::integral_constant<int, 8>{});
        else go(l, std::integral_constant<int, 16>{});
      };
      if (lanes == 16) by_slots(std::integral_constant<int, 16>{});
      else by_slots(std::integral_constant<int, 64>{});
      return launch_status("moe_route");
    }
  }
  by_width(L.E, [&](auto epl) {
    if (L.bf16) hipLaunchKernelGGL((k_route<1, epl.value>), token_grid(L.T), 256, 0, st, a);
    else hipLaunchKernelGGL((k_route<0, epl.value>), token_grid(L.T), 256, 0, st, a);
  });
  return launch_status("moe_route");
}

static bsq_status route_backward_part(const RouteBackwardLaunch& L, hipStream_t st) {
  const RouteBwdArgs a{L.T, L.E, L.k, L.logits, L.sigmoid, L.renorm, L.scale, L.ids, L.dweights, L.dscores,
                       L.dlogits};
  if (L.E <= 256 && L.k <= 16 && L.T >= kRowTokens) {
    const unsigned grid = unsigned((L.T + 15) / 16);
    auto go = [&](auto s) {
      if (L.bf16) hipLaunchKernelGGL((k_route_backward_rows<1, s.value>), grid, 256, 0, st, a);
      else hipLaunchKernelGGL((k_route_backward_rows<0, s.value>), grid, 256, 0, st, a);
    };
    if (L.E <= 64) go(std::integral_constant<int, 4>{});
    else if (L.E <= 128) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 16>{});
    return launch_status("moe_route_backward");
  }
  by_width(L.E, [&](auto epl) {
    if (L.bf16) hipLaunchKernelGGL((k_route_backward<1, epl.value>), token_grid(L.T), 256, 0, st, a);
    else hipLaunchKernelGGL((k_route_backward<0, epl.value>), token_grid(L.T), 256, 0, st, a);
  });
  return launch_status("moe_route_backward");
}

static const void* logits_from(const void* p, bool bf16, int64_t elem) {
  return static_cast<const char*>(p) + elem * (bf16 ? 2 : 4);
}

bsq_status launch_route(const RouteLaunch& L, hipStream_t st) {
  return in_parts(L.T, kLaunchTokens, [&](int64_t t, int64_t n) {
    RouteLaunch P = L;
    P.T = n;
    P.logits = logits_from(L.logits, L.bf16, t * L.E);
    P.ids += t * L.k;
    P.weights += t * L.k;
    if (L.scores != nullptr) P.scores += t * L.E;
    return route_part(P, st);
  });
}

bsq_status launch_route_backward(const RouteBackwardLaunch& L, hipStream_t st) {
  return in_parts(L.T, kLaunchTokens, [&](int64_t t, int64_t n) {
    RouteBackwardLaunch P = L;
    P.T = n;
    P.logits = logits_from(L.logits, L.bf16, t * L.E);
    P.ids += t * L.k;
    P.dweights += t * L.k;
    if (L.dscores != nullptr) P.dscores += t * L.E;
    P.dlogits = const_cast<void*>(logits_from(L.dlogits, L.bf16, t * L.E));
    return route_backward_part(P, st);
  });
}

}  // namespace bsq
