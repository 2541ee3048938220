// Launcher of the products with 4-bit weights (arguments already validated).
#pragma once

#include "common.h"
#include "moe_index.h"

namespace bsq {

enum class Code4 { e4m3, e5m2, e2m1 };  // of A

struct Mx4Launch {
  int64_t T;    // rows of A (dense: of each product of the batch)
  int64_t cap;  // rows of out (dense: T)
  int64_t E;    // experts (dense: products of the batch)
  int k;
  int64_t N, K;
  const uint8_t *A, *SA;  // [T, K] codes or [T, K / 2] packed (dense: [E, T, ..])
  const uint8_t *B, *SB;  // [E, N, K / 2], [E, N, K / 32]
  const int32_t* offsets;  // [E + 1]; null: dense
  const int32_t* rows;     // [cap] or null
  void* out;               // [cap, N] (dense: [E, T, N])
  Code4 a;
  bool out_bf16;
};
bsq_status launch_mx4_product(const Mx4Launch& L, hipStream_t st);

}  // namespace bsq
