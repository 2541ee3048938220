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
#include <math.h>

#include "moe.h"

namespace bsq {

namespace {

constexpr int kRouteMaxE = 1024;

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
      p[i] = top == -INFINITY ? 0.0 : exp(p[i] - top);
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
  double w_mine = 0.0, total = 0.0;
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
    total += pb;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id_mine;
    const double w = a.renorm ? (total == 0.0 ? 0.0 : w_mine / total) : w_mine;
    a.weights[t * a.k + lane] = float(w * double(a.scale));
  }
}

template <int BF16, int EPL>
__global__ void __launch_bounds__(256) k_route(RouteArgs a) {
  __shared__ double cs[4][64 * EPL];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t t = int64_t(blockIdx.x) * 4 + w; t < a.T; t += int64_t(gridDim.x) * 4)
    route_token<BF16, EPL>(a, t, lane, cs[w]);
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

// With total = the sum of the chosen p: dp at a choice is
// scale (dw - sum(dw p) / total) / total where renormalised, else scale dw,
// plus dscores; softmax dx = p (dp - sum p dp), sigmoid dx = dp p (1 - p).
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
      p[i] = top == -INFINITY ? 0.f : expf(p[i] - top);
      sum += p[i];
    }
    sum = wave_sum(sum);
    const float r = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= r;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) dps[lane + 64 * i] = p[i];
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
  const bool on = id >= 0 && id < E;
  const float pc = on ? dps[id] : 0.f;
  float d = on ? a.dweights[t * a.k + lane] * a.scale : 0.f;
  if (a.renorm) {
    const float total = wave_sum(pc);
    const float r = total == 0.f ? 0.f : 1.0f / total;
    d = (d - wave_sum(d * (pc * r))) * r;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < EPL; ++i) dps[lane + 64 * i] = 0.f;
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  if (on) dps[id] = d;
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    dp[i] = dps[e];
    if (a.dscores != nullptr && e < E) dp[i] += a.dscores[t * E + e];
    if (e < E) dot += p[i] * dp[i];
  }
  __builtin_amdgcn_wave_barrier();
  if (!a.sigmoid) dot = wave_sum(dot);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < E) {
      const float dx = a.sigmoid ? dp[i] * p[i] * q[i] : p[i] * (dp[i] - dot);
      if (BF16)
        static_cast<uint16_t*>(a.dlogits)[t * E + e] = uint16_t(encode_bf16(dx));
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

template <typename F>
void by_width(int E, F&& f) {
  const int epl = (E + 63) / 64;
  if (epl <= 1) f(std::integral_constant<int, 1>{});
  else if (epl <= 2) f(std::integral_constant<int, 2>{});
  else if (epl <= 4) f(std::integral_constant<int, 4>{});
  else if (epl <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

unsigned token_grid(int64_t T) {
  const int64_t g = (T + 3) / 4;
  return unsigned(g < 65536 ? g : 65536);
}

}  // namespace

bsq_status launch_route(const RouteLaunch& L, hipStream_t st) {
  const RouteArgs a{L.T, L.E, L.k, L.groups, L.top_groups, L.group_top, L.logits, L.sigmoid, L.renorm, L.scale,
                    L.bias, L.ids, L.weights, L.scores};
  by_width(L.E, [&](auto epl) {
    if (L.bf16) hipLaunchKernelGGL((k_route<1, epl.value>), token_grid(L.T), 256, 0, st, a);
    else hipLaunchKernelGGL((k_route<0, epl.value>), token_grid(L.T), 256, 0, st, a);
  });
  return launch_status("moe_route");
}

bsq_status launch_route_backward(const RouteBackwardLaunch& L, hipStream_t st) {
  const RouteBwdArgs a{L.T, L.E, L.k, L.logits, L.sigmoid, L.renorm, L.scale, L.ids, L.dweights, L.dscores,
                       L.dlogits};
  by_width(L.E, [&](auto epl) {
    if (L.bf16) hipLaunchKernelGGL((k_route_backward<1, epl.value>), token_grid(L.T), 256, 0, st, a);
    else hipLaunchKernelGGL((k_route_backward<0, epl.value>), token_grid(L.T), 256, 0, st, a);
  });
  return launch_status("moe_route_backward");
}

}  // namespace bsq
