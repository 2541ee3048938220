// The C ABI of the calls on 4-bit operands (declared in include/bsq.h):
// argument validation on the host, then kernel launches on the caller's stream.
#include "common.h"
#include "gemm4.h"
#include "norm.h"
#include "quant4.h"

using namespace bsq;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 60;
constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxContraction = int64_t(1) << 24;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxNorm = int64_t(1) << 24;  // values of a row

bool elems_fit(int64_t a, int64_t b, int64_t c = 1) {
  int64_t n = 0;
  return !__builtin_mul_overflow(a, b, &n) && !__builtin_mul_overflow(n, c, &n) && n <= kMaxElems;
}
bool is_wide(int d) { return d == BSQ_F32 || d == BSQ_BF16; }
bool is_code(int d) { return d == BSQ_E4M3 || d == BSQ_E5M2 || d == BSQ_E2M1; }
bool known_dtype(int d) { return d >= BSQ_F32 && d <= BSQ_E2M1; }
bool word(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }
Code4 code_of(int d) { return d == BSQ_E4M3 ? Code4::e4m3 : d == BSQ_E5M2 ? Code4::e5m2 : Code4::e2m1; }

#define BSQ_DEVICE()                       \
  do {                                     \
    bsq_status _s = require_gfx950();      \
    if (_s != BSQ_OK) return _s;           \
  } while (0)

}  // namespace

extern "C" {

// --------------------------------------------------------------- quantizer --

bsq_status bsq_quant_fp4(int64_t B, int64_t rows, int64_t cols, const void* src, int src_dtype, int format,
                         const float* factor, uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                         void* stream) {
  BSQ_CHECK(B >= 0 && rows >= 0 && cols >= 0, BSQ_ERR_SHAPE, "negative size");
  BSQ_CHECK(elems_fit(B, rows, cols), BSQ_ERR_UNSUPPORTED, "more than 2^60 elements");
  BSQ_CHECK(known_dtype(src_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(format == BSQ_MXFP4 || format == BSQ_NVFP4, BSQ_ERR_DTYPE, "unknown format");
  BSQ_CHECK(is_wide(src_dtype), BSQ_ERR_UNSUPPORTED, "src must be F32 or BF16");
  BSQ_CHECK(factor == nullptr || format == BSQ_NVFP4, BSQ_ERR_UNSUPPORTED, "a factor is for NVFP4 only");
  const int64_t block = format == BSQ_NVFP4 ? 16 : 32;
  BSQ_CHECK(cols % block == 0, BSQ_ERR_SHAPE, "cols must be a multiple of the block (32, NVFP4 16)");
  BSQ_CHECK(codes_t == nullptr || rows % block == 0, BSQ_ERR_SHAPE,
            "rows must be a multiple of the block (32, NVFP4 16) for the transposed codes");
  BSQ_CHECK((codes == nullptr) == (scales == nullptr) && (codes_t == nullptr) == (scales_t == nullptr), BSQ_ERR_NULL,
            "codes and their scales come together");
  if (B == 0 || rows == 0 || cols == 0 || (codes == nullptr && codes_t == nullptr)) return ok();
  // tiles of 128 x 128, numbered in 64 bits along rows and columns of 32
  BSQ_CHECK((rows + 127) / 128 <= kMaxInt && (cols + 127) / 128 <= kMaxInt / 2, BSQ_ERR_UNSUPPORTED,
            "more than 2^31 - 1 rows of tiles, or 2^30 - 1 columns");
  BSQ_CHECK_PTR(src);
  BSQ_CHECK(aligned16(codes) && aligned16(codes_t), BSQ_ERR_ALIGN, "codes not 16-byte aligned");
  BSQ_CHECK(word(factor), BSQ_ERR_ALIGN, "factor is not 4-byte aligned");
  BSQ_DEVICE();
  return launch_quant4(Quant4Launch{B, rows, cols, src, src_dtype == BSQ_BF16, format == BSQ_NVFP4, factor, codes,
                                    scales, codes_t, scales_t},
                       as_stream(stream));
}

// ---------------------------------------------------------------- products --

static bsq_status product_check(int64_t E, int64_t T, int64_t N, int64_t K, int a_dtype, int out_dtype) {
  BSQ_CHECK(known_dtype(a_dtype) && known_dtype(out_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(K % 32 == 0, BSQ_ERR_SHAPE, "K must be a multiple of the block (32)");
  BSQ_CHECK(is_code(a_dtype), BSQ_ERR_UNSUPPORTED, "the left operand must be E2M1, E4M3 or E5M2");
  BSQ_CHECK(is_wide(out_dtype), BSQ_ERR_UNSUPPORTED, "out_dtype must be F32 or BF16");
  BSQ_CHECK(N % 16 == 0, BSQ_ERR_UNSUPPORTED, "the library needs N % 16 == 0");
  BSQ_CHECK(T <= (int64_t(1) << 30) && N <= (int64_t(1) << 30) && K <= kMaxContraction, BSQ_ERR_UNSUPPORTED,
            "extent too large");
  // scales are addressed with 32-bit byte offsets inside a product
  BSQ_CHECK(elems_fit(E, N, K) && elems_fit(E, T, K) && T * (K / 32) <= int64_t(0xFFFFFFF0) &&
                N * (K / 32) <= int64_t(0xFFFFFFF0),
            BSQ_ERR_UNSUPPORTED, "an operand too large");
  return BSQ_OK;
}

bsq_status bsq_scaled_matmul_mxfp4(int64_t B, int64_t M, int64_t N, int64_t K, const uint8_t* lhs, int lhs_dtype,
                                   const uint8_t* rhs, const uint8_t* lhs_scales, const uint8_t* rhs_scales,
                                   void* out, int out_dtype, void* stream) {
  BSQ_CHECK(B >= 0 && M >= 0 && N >= 0 && K >= 0, BSQ_ERR_SHAPE, "negative size");
  const bsq_status s = product_check(B, M, N, K, lhs_dtype, out_dtype);
  if (s != BSQ_OK) return s;
  BSQ_CHECK(B <= kMaxBatch, BSQ_ERR_UNSUPPORTED, "batch over 65535");
  BSQ_CHECK(elems_fit(B, M, N) && B * ((M + 15) / 16) <= kMaxInt / ((N + 15) / 16 + 1), BSQ_ERR_UNSUPPORTED,
            "more than 2^31 - 1 tiles of 16 x 16");
  if (B == 0 || M == 0 || N == 0) return ok();
  BSQ_CHECK_PTR(out);
  if (K > 0) {
    BSQ_CHECK_PTR(lhs);
    BSQ_CHECK_PTR(rhs);
    BSQ_CHECK(lhs_scales != nullptr && rhs_scales != nullptr, BSQ_ERR_NULL, "scales are NULL");
    BSQ_CHECK(word(lhs_scales) && word(rhs_scales), BSQ_ERR_ALIGN, "scales must be 4-byte aligned");
  }
  BSQ_DEVICE();
  return launch_mx4_product(Mx4Launch{M, M, B, 1, N, K, lhs, lhs_scales, rhs, rhs_scales, nullptr, nullptr, out,
                                      code_of(lhs_dtype), out_dtype == BSQ_BF16},
                            as_stream(stream));
}

bsq_status bsq_moe_matmul_mxfp4(int64_t T, int64_t cap, int64_t E, int64_t N, int64_t K, int64_t k, const uint8_t* a,
                                int a_dtype, const uint8_t* a_scales, const uint8_t* b, const uint8_t* b_scales,
                                const int32_t* offsets, const int32_t* rows, void* out, int out_dtype,
                                void* stream) {
  BSQ_CHECK(T >= 0 && cap >= 0 && E >= 1 && N >= 0 && K >= 0 && k >= 1, BSQ_ERR_SHAPE,
            "negative size, or E or k below 1");
  const bsq_status s = product_check(E, T, N, K, a_dtype, out_dtype);
  if (s != BSQ_OK) return s;
  BSQ_CHECK(E <= kMaxExperts, BSQ_ERR_UNSUPPORTED, "at most 1024 experts");
  BSQ_CHECK(cap <= kMaxRows && k <= kMaxInt, BSQ_ERR_UNSUPPORTED, "extent too large");
  BSQ_CHECK(elems_fit(cap, N) && cap / 16 + E + 1 <= kMaxInt / ((N + 15) / 16 + 1), BSQ_ERR_UNSUPPORTED,
            "more than 2^31 - 1 tiles of 16 x 16");
  if (cap == 0 || N == 0) return ok();
  BSQ_CHECK_PTR(out);
  BSQ_CHECK_PTR(offsets);
  BSQ_CHECK(aligned16(rows), BSQ_ERR_ALIGN, "rows is not 16-byte aligned");
  if (K > 0 && T > 0) {
    BSQ_CHECK_PTR(a);
    BSQ_CHECK_PTR(b);
    BSQ_CHECK(a_scales != nullptr && b_scales != nullptr, BSQ_ERR_NULL, "scales are NULL");
    BSQ_CHECK(word(a_scales) && word(b_scales), BSQ_ERR_ALIGN, "scales must be 4-byte aligned");
  }
  BSQ_DEVICE();
  return launch_mx4_product(Mx4Launch{T, cap, E, int(k), N, K, a, a_scales, b, b_scales, offsets, rows, out,
                                      code_of(a_dtype), out_dtype == BSQ_BF16},
                            as_stream(stream));
}

// -------------------------------------------------------------------- norm --

static bsq_status norm_check(int64_t R, int64_t C, int dtype, int kind) {
  BSQ_CHECK(R >= 0 && C >= 0, BSQ_ERR_SHAPE, "negative size");
  BSQ_CHECK(elems_fit(R, C), BSQ_ERR_UNSUPPORTED, "more than 2^60 elements");
  BSQ_CHECK(known_dtype(dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(kind == BSQ_LAYER_NORM || kind == BSQ_RMS_NORM, BSQ_ERR_DTYPE, "unknown kind of norm");
  BSQ_CHECK(is_wide(dtype), BSQ_ERR_UNSUPPORTED, "x must be F32 or BF16");
  BSQ_CHECK(C <= kMaxNorm, BSQ_ERR_UNSUPPORTED, "rows of more than 2^24 values");
  return BSQ_OK;
}

bsq_status bsq_norm_mx(int64_t R, int64_t C, const void* x, int x_dtype, int kind, float eps, const float* gamma,
                       const float* beta, void* y, int code_dtype, uint8_t* codes, uint8_t* scales, float* mean,
                       float* rstd, void* stream) {
  const bsq_status s = norm_check(R, C, x_dtype, kind);
  if (s != BSQ_OK) return s;
  BSQ_CHECK((codes == nullptr) == (scales == nullptr), BSQ_ERR_NULL, "codes and their scales come together");
  if (codes != nullptr) {
    BSQ_CHECK(known_dtype(code_dtype), BSQ_ERR_DTYPE, "unknown dtype");
    BSQ_CHECK(is_code(code_dtype), BSQ_ERR_UNSUPPORTED, "code_dtype must be E4M3, E5M2 or E2M1");
    BSQ_CHECK(C % 32 == 0, BSQ_ERR_SHAPE, "C must be a multiple of the block (32) for codes");
  }
  BSQ_CHECK(eps >= 0.0f, BSQ_ERR_UNSUPPORTED, "eps must not be negative");
  if (R == 0 || C == 0) return ok();
  BSQ_CHECK_PTR(x);
  BSQ_CHECK(aligned16(y) && aligned16(codes) && aligned16(gamma) && aligned16(beta), BSQ_ERR_ALIGN,
            "y, codes, gamma or beta not 16-byte aligned");
  BSQ_CHECK(word(mean) && word(rstd), BSQ_ERR_ALIGN, "mean or rstd not 4-byte aligned");
  BSQ_DEVICE();
  const NormCode code = codes == nullptr         ? NormCode::none
                        : code_dtype == BSQ_E4M3 ? NormCode::e4m3
                        : code_dtype == BSQ_E5M2 ? NormCode::e5m2
                                                 : NormCode::e2m1;
  return launch_norm(NormLaunch{R, C, x, x_dtype == BSQ_BF16, kind == BSQ_RMS_NORM, eps, gamma, beta, y, code, codes,
                                scales, mean, rstd},
                     as_stream(stream));
}

size_t bsq_norm_backward_workspace_bytes(int64_t R, int64_t C) {
  if (R < 0 || C < 0) return 0;
  if (C > kMaxNorm) return SIZE_MAX;
  const size_t b = size_t(8) * size_t(C) * size_t(R < kNormGroups ? R : kNormGroups);
  return b < 16 ? 16 : b;
}

bsq_status bsq_norm_backward(int64_t R, int64_t C, const void* x, const void* dy, int x_dtype, int kind,
                             const float* gamma, const float* mean, const float* rstd, void* dx, float* dgamma,
                             float* dbeta, void* workspace, size_t workspace_bytes, void* stream) {
  const bsq_status s = norm_check(R, C, x_dtype, kind);
  if (s != BSQ_OK) return s;
  const bool weights = dgamma != nullptr || dbeta != nullptr;
  BSQ_CHECK(!weights || workspace_bytes >= bsq_norm_backward_workspace_bytes(R, C), BSQ_ERR_SHAPE,
            "workspace too small");
  if (C == 0 || (R == 0 && !weights)) return ok();
  if (R > 0) {
    BSQ_CHECK_PTR(x);
    BSQ_CHECK_PTR(dy);
    BSQ_CHECK_PTR(dx);
    BSQ_CHECK(rstd != nullptr && (mean != nullptr || kind == BSQ_RMS_NORM), BSQ_ERR_NULL, "mean or rstd is NULL");
    BSQ_CHECK(word(mean) && word(rstd), BSQ_ERR_ALIGN, "mean or rstd not 4-byte aligned");
    if (weights) BSQ_CHECK_PTR(workspace);
  }
  BSQ_CHECK(aligned16(gamma) && word(dgamma) && word(dbeta), BSQ_ERR_ALIGN, "gamma, dgamma or dbeta not aligned");
  BSQ_DEVICE();
  return launch_norm_backward(NormBackwardLaunch{R, C, x, dy, x_dtype == BSQ_BF16, kind == BSQ_RMS_NORM, gamma, mean,
                                                 rstd, dx, dgamma, dbeta, static_cast<float*>(workspace)},
                              as_stream(stream));
}

}  // extern "C"
