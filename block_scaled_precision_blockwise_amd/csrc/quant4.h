// Launcher of the quantizer to 4-bit codes (arguments already validated).
#pragma once

#include "common.h"

namespace bsq {

struct Quant4Launch {
  int64_t B, R, C;
  const void* src;      // [B, R, C]
  bool bf16;            // else float32
  bool nv;              // nvfp4 (blocks of 16, E4M3 scales), else mxfp4 (32, E8M0)
  const float* factor;  // [1] or null
  uint8_t *codes, *scales;      // [B, R, C / 2], [B, R, C / block], or null
  uint8_t *codes_t, *scales_t;  // [B, C, R / 2], [B, C, R / block], or null
};
bsq_status launch_quant4(const Quant4Launch& L, hipStream_t st);

}  // namespace bsq
