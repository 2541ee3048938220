// Launchers of the expert-layer kernels (arguments already validated).
#pragma once

#include "common.h"

namespace bsq {

// ----------------------------------------------------------------- route --
struct RouteLaunch {
  int64_t T;
  int E, k;
  int groups, top_groups, group_top;
  const void* logits;  // [T, E]
  bool bf16;           // logits (and dlogits) are bfloat16, else float32
  bool sigmoid;        // else softmax
  bool renorm;
  float scale;
  const float* bias;   // [E] or null
  int32_t* ids;        // [T, k]
  float* weights;      // [T, k]
  float* scores;       // [T, E] or null
};
bsq_status launch_route(const RouteLaunch& L, hipStream_t st);

struct RouteBackwardLaunch {
  int64_t T;
  int E, k;
  const void* logits;
  bool bf16, sigmoid, renorm;
  float scale;
  const int32_t* ids;
  const float* dweights;  // [T, k]
  const float* dscores;   // [T, E] or null
  void* dlogits;          // [T, E], type of logits
};
bsq_status launch_route_backward(const RouteBackwardLaunch& L, hipStream_t st);

// ------------------------------------------------------------------ rows --
// Workgroups (and rows of the workspace's counts) that n choices are dealt to.
int plan_blocks(int64_t n);
bsq_status launch_plan(int64_t n, int E, int align, int64_t cap, const int32_t* ids, int32_t* offsets,
                       int32_t* counts, int32_t* rows, int32_t* pos, int32_t* space, hipStream_t st);
bsq_status launch_gather_mx(int64_t T, int64_t H, int64_t cap, int k, const void* x, bool bf16, const int32_t* rows,
                            const float* weights, bool e5m2, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                            uint8_t* scales_t, hipStream_t st);
bsq_status launch_combine(int64_t T, int64_t H, int64_t cap, int k, const void* y, bool bf16, const int32_t* pos,
                          const float* weights, void* out, hipStream_t st);
bsq_status launch_combine_backward(int64_t T, int64_t H, int64_t cap, int k, const void* y, bool bf16,
                                   const int32_t* pos, const void* dout, float* dweights, hipStream_t st);

// -------------------------------------------------------------- products --
struct MoeGemmLaunch {
  int64_t T;             // rows of A
  int64_t cap;           // rows of out (product) / contraction length (wgrad)
  int E, k;
  int64_t N, K;
  const uint8_t* A;      // product [T, K]; wgrad dyt [N, cap]
  const uint8_t* SA;
  const uint8_t* B;      // product [E, N, K]; wgrad xt [K, cap]
  const uint8_t* SB;
  const int32_t* offsets;  // [E + 1]
  const int32_t* rows;     // [cap] or null (row r of out takes row r of A)
  void* out;               // product [cap, N]; wgrad [E, N, K]
  bool a_e5m2, out_bf16;
};
bsq_status launch_moe_product(const MoeGemmLaunch& L, hipStream_t st);
bsq_status launch_moe_wgrad(const MoeGemmLaunch& L, hipStream_t st);

// ------------------------------------------------------------------ gate --
bsq_status launch_swiglu_mx(int64_t R, int64_t F, const void* gu, bool bf16, bool e5m2, uint8_t* h, uint8_t* h_scales,
                            uint8_t* ht, uint8_t* ht_scales, uint8_t* kept, uint8_t* kept_scales, hipStream_t st);
bsq_status launch_swiglu_mx_backward(int64_t R, int64_t F, const uint8_t* kept, const uint8_t* kept_scales, bool e5m2,
                                     const void* dh, bool bf16, void* dgu, hipStream_t st);

}  // namespace bsq
