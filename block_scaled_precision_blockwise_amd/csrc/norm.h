// Launchers of the norm and its gradient (arguments already validated).
#pragma once

#include "common.h"

namespace bsq {

enum class NormCode { none, e4m3, e5m2, e2m1 };

struct NormLaunch {
  int64_t R, C;
  const void* x;
  bool bf16;  // x and y, else float32
  bool rms;   // no mean is taken off
  float eps;
  const float *gamma, *beta;  // [C] or null
  void* y;                    // [R, C] or null
  NormCode code;
  uint8_t *codes, *scales;  // or null
  float *mean, *rstd;       // [R] or null
};
bsq_status launch_norm(const NormLaunch& L, hipStream_t st);

// Rows of partial sums that the workspace has at most.
constexpr int64_t kNormGroups = 1024;

struct NormBackwardLaunch {
  int64_t R, C;
  const void *x, *dy;
  bool bf16, rms;
  const float *gamma;         // [C] or null
  const float *mean, *rstd;   // [R]; mean null with rms
  void* dx;                   // [R, C]
  float *dgamma, *dbeta;      // [C] or null
  float* space;               // [2, groups, C]
};
bsq_status launch_norm_backward(const NormBackwardLaunch& L, hipStream_t st);

}  // namespace bsq
