// The C ABI of the expert-layer calls (declared in include/bsq.h): argument
// validation on the host, then kernel launches on the caller's stream.
#include <climits>

#include "common.h"
#include "moe.h"
#include "moe_index.h"

using namespace bsq;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 60;
constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxContraction = int64_t(1) << 24;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxChoices = 64;  // of one token

bool elems_fit(int64_t a, int64_t b, int64_t c = 1) {
  int64_t n = 0;
  return !__builtin_mul_overflow(a, b, &n) && !__builtin_mul_overflow(n, c, &n) && n <= kMaxElems;
}
bool is_fp8(int d) { return d == BSQ_E4M3 || d == BSQ_E5M2; }
bool is_wide(int d) { return d == BSQ_F32 || d == BSQ_BF16; }
bool known_dtype(int d) { return d >= BSQ_F32 && d <= BSQ_I32; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

#define BSQ_DEVICE()                       \
  do {                                     \
    bsq_status _s = require_gfx950();      \
    if (_s != BSQ_OK) return _s;           \
  } while (0)

// Rows that n choices over E experts take at most, each segment rounded up
// to `align` rows; -1 where that passes 64 bits.
int64_t capacity(int64_t n, int64_t E, int64_t align) {
  int64_t pad = 0, c = 0;
  if (__builtin_mul_overflow(n < E ? n : E, align - 1, &pad) || __builtin_add_overflow(n, pad, &c)) return -1;
  return c;
}

}  // namespace

extern "C" {

// ----------------------------------------------------------------- routing --

bsq_status bsq_moe_route(int64_t T, int64_t E, int64_t k, int64_t groups, int64_t top_groups, int64_t group_top,
                         const void* logits, int logits_dtype, const float* bias, int score, int renorm, float scale,
                         int32_t* ids, float* weights, float* scores, void* stream) {
  BSQ_CHECK(T >= 0 && E >= 1 && k >= 1, BSQ_ERR_SHAPE, "negative T, or E or k below 1");
  BSQ_CHECK(groups >= 1 && top_groups >= 1 && top_groups <= groups && E % groups == 0, BSQ_ERR_SHAPE,
            "E must be a multiple of groups, and 1 <= top_groups <= groups");
  BSQ_CHECK(group_top >= 1 && group_top <= E / groups, BSQ_ERR_SHAPE, "group_top must be 1 .. E / groups");
  BSQ_CHECK(k <= top_groups * (E / groups), BSQ_ERR_SHAPE, "k exceeds the experts of top_groups groups");
  BSQ_CHECK(known_dtype(logits_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(score == BSQ_SOFTMAX || score == BSQ_SIGMOID, BSQ_ERR_DTYPE, "unknown score");
  BSQ_CHECK(is_wide(logits_dtype), BSQ_ERR_UNSUPPORTED, "logits must be F32 or BF16");
  BSQ_CHECK(E <= kMaxExperts && k <= kMaxChoices && groups <= 64 && group_top <= 2, BSQ_ERR_UNSUPPORTED,
            "at most 1024 experts, 64 choices, 64 groups, group_top 2");
  BSQ_CHECK(T <= kMaxInt, BSQ_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens");
  if (T == 0) return ok();
  BSQ_CHECK_PTR(logits);
  BSQ_CHECK_PTR(ids);
  BSQ_CHECK_PTR(weights);
  BSQ_CHECK(aligned16(bias) && aligned16(scores), BSQ_ERR_ALIGN, "bias or scores is not 16-byte aligned");
  BSQ_DEVICE();
  const RouteLaunch L{T,      int(E), int(k), int(groups), int(top_groups), int(group_top), logits, logits_dtype == BSQ_BF16,
                      score == BSQ_SIGMOID, renorm != 0, scale, bias, ids, weights, scores};
  return launch_route(L, as_stream(stream));
}

bsq_status bsq_moe_route_backward(int64_t T, int64_t E, int64_t k, const void* logits, int logits_dtype, int score,
                                  int renorm, float scale, const int32_t* ids, const float* dweights,
                                  const float* dscores, void* dlogits, void* stream) {
  BSQ_CHECK(T >= 0 && E >= 1 && k >= 1 && k <= E, BSQ_ERR_SHAPE, "negative T, E below 1, or k outside 1 .. E");
  BSQ_CHECK(known_dtype(logits_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(score == BSQ_SOFTMAX || score == BSQ_SIGMOID, BSQ_ERR_DTYPE, "unknown score");
  BSQ_CHECK(is_wide(logits_dtype), BSQ_ERR_UNSUPPORTED, "logits must be F32 or BF16");
  BSQ_CHECK(E <= kMaxExperts && k <= kMaxChoices, BSQ_ERR_UNSUPPORTED, "at most 1024 experts, 64 choices");
  BSQ_CHECK(T <= kMaxInt, BSQ_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens");
  if (T == 0) return ok();
  BSQ_CHECK_PTR(logits);
  BSQ_CHECK_PTR(ids);
  BSQ_CHECK_PTR(dweights);
  BSQ_CHECK_PTR(dlogits);
  BSQ_CHECK(aligned16(dscores), BSQ_ERR_ALIGN, "dscores is not 16-byte aligned");
  BSQ_DEVICE();
  const RouteBackwardLaunch L{T,      int(E), int(k), logits, logits_dtype == BSQ_BF16, score == BSQ_SIGMOID, renorm != 0,
                              scale, ids,    dweights, dscores, dlogits};
  return launch_route_backward(L, as_stream(stream));
}

// -------------------------------------------------------------------- rows --

int64_t bsq_moe_capacity(int64_t n, int64_t E, int64_t align) {
  if (n < 0 || E < 1 || align < 1) return 0;
  const int64_t c = capacity(n, E, align);
  if (c < 0 || c > kMaxElems || align > kMaxElems) return INT64_MAX;
  return (c + align - 1) / align * align;
}

size_t bsq_moe_plan_workspace_bytes(int64_t n, int64_t E) {
  if (n < 0 || E < 1) return 0;
  if (n > kMaxInt || E > kMaxExperts) return SIZE_MAX;
  const size_t b = size_t(4) * size_t(E) * size_t(plan_blocks(n) + 1);
  return b < 16 ? 16 : b;
}

bsq_status bsq_moe_plan(int64_t n, int64_t E, int64_t align, int64_t cap, const int32_t* ids, int32_t* offsets,
                        int32_t* counts, int32_t* rows, int32_t* pos, void* workspace, size_t workspace_bytes,
                        void* stream) {
  BSQ_CHECK(n >= 0 && E >= 1 && align >= 1 && cap >= 0, BSQ_ERR_SHAPE, "negative n or cap, or E or align below 1");
  BSQ_CHECK(n <= kMaxInt && cap <= kMaxInt && align <= kMaxInt, BSQ_ERR_UNSUPPORTED, "n, cap or align over 2^31 - 1");
  BSQ_CHECK(E <= kMaxExperts, BSQ_ERR_UNSUPPORTED, "at most 1024 experts");
  const int64_t need = capacity(n, E, align);
  BSQ_CHECK(need >= 0 && cap >= need, BSQ_ERR_SHAPE, "fewer rows than n + min(E, n) (align - 1)");
  BSQ_CHECK(workspace_bytes >= bsq_moe_plan_workspace_bytes(n, E), BSQ_ERR_SHAPE, "workspace too small");
  BSQ_CHECK_PTR(offsets);
  BSQ_CHECK_PTR(counts);
  if (cap > 0) BSQ_CHECK_PTR(rows);
  if (n > 0) {
    BSQ_CHECK_PTR(ids);
    BSQ_CHECK_PTR(pos);
    BSQ_CHECK_PTR(workspace);
  }
  BSQ_DEVICE();
  return launch_plan(n, int(E), int(align), cap, ids, offsets, counts, rows, pos, static_cast<int32_t*>(workspace),
                     as_stream(stream));
}

bsq_status bsq_moe_gather_mx(int64_t T, int64_t H, int64_t cap, int64_t k, const void* x, int x_dtype,
                             const int32_t* rows, const float* weights, int code_dtype, uint8_t* codes,
                             uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  BSQ_CHECK(T >= 0 && H >= 0 && cap >= 0 && k >= 1, BSQ_ERR_SHAPE, "negative size, or k below 1");
  BSQ_CHECK(elems_fit(T, H) && elems_fit(cap, H), BSQ_ERR_UNSUPPORTED, "more than 2^60 elements");
  BSQ_CHECK(known_dtype(x_dtype) && known_dtype(code_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(is_wide(x_dtype), BSQ_ERR_UNSUPPORTED, "x must be F32 or BF16");
  BSQ_CHECK(is_fp8(code_dtype), BSQ_ERR_UNSUPPORTED, "code_dtype must be E4M3 or E5M2");
  BSQ_CHECK(H % 32 == 0, BSQ_ERR_SHAPE, "H must be a multiple of 32");
  BSQ_CHECK(codes_t == nullptr || cap % 32 == 0, BSQ_ERR_SHAPE, "cap must be a multiple of 32 for the transposed codes");
  BSQ_CHECK(cap <= kMaxInt && k <= kMaxInt, BSQ_ERR_UNSUPPORTED, "cap or k over 2^31 - 1");
  BSQ_CHECK(((cap + 127) / 128) * ((H + 63) / 64) <= kMaxInt, BSQ_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles");
  BSQ_CHECK((codes == nullptr) == (scales == nullptr) && (codes_t == nullptr) == (scales_t == nullptr), BSQ_ERR_NULL,
            "codes and their scales come together");
  if (cap == 0 || H == 0 || (codes == nullptr && codes_t == nullptr)) return ok();
  if (T > 0) BSQ_CHECK_PTR(x);
  BSQ_CHECK_PTR(rows);
  BSQ_CHECK(aligned16(codes) && aligned16(codes_t) && aligned16(weights), BSQ_ERR_ALIGN,
            "codes or weights not 16-byte aligned");
  BSQ_DEVICE();
  return launch_gather_mx(T, H, cap, int(k), x, x_dtype == BSQ_BF16, rows, weights, code_dtype == BSQ_E5M2, codes,
                          scales, codes_t, scales_t, as_stream(stream));
}

static bsq_status combine_check(int64_t T, int64_t H, int64_t cap, int64_t k, int y_dtype) {
  BSQ_CHECK(T >= 0 && H >= 0 && cap >= 0 && k >= 1, BSQ_ERR_SHAPE, "negative size, or k below 1");
  BSQ_CHECK(elems_fit(T, H) && elems_fit(cap, H) && elems_fit(T, k), BSQ_ERR_UNSUPPORTED, "more than 2^60 elements");
  BSQ_CHECK(known_dtype(y_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(is_wide(y_dtype), BSQ_ERR_UNSUPPORTED, "y must be F32 or BF16");
  BSQ_CHECK(H % 8 == 0, BSQ_ERR_SHAPE, "H must be a multiple of 8");
  BSQ_CHECK(k <= kMaxInt && T <= kMaxInt && cap <= kMaxInt, BSQ_ERR_UNSUPPORTED, "T, k or cap over 2^31 - 1");
  return BSQ_OK;
}

bsq_status bsq_moe_combine(int64_t T, int64_t H, int64_t cap, int64_t k, const void* y, int y_dtype,
                           const int32_t* pos, const float* weights, void* out, void* stream) {
  const bsq_status s = combine_check(T, H, cap, k, y_dtype);
  if (s != BSQ_OK) return s;
  if (T == 0 || H == 0) return ok();
  if (cap > 0) BSQ_CHECK_PTR(y);
  BSQ_CHECK_PTR(pos);
  BSQ_CHECK_PTR(out);
  BSQ_CHECK(aligned16(weights), BSQ_ERR_ALIGN, "weights is not 16-byte aligned");
  BSQ_DEVICE();
  return launch_combine(T, H, cap, int(k), y, y_dtype == BSQ_BF16, pos, weights, out, as_stream(stream));
}

bsq_status bsq_moe_combine_backward(int64_t T, int64_t H, int64_t cap, int64_t k, const void* y, int y_dtype,
                                    const int32_t* pos, const void* dout, float* dweights, void* stream) {
  const bsq_status s = combine_check(T, H, cap, k, y_dtype);
  if (s != BSQ_OK) return s;
  if (T == 0) return ok();
  if (H > 0) {
    if (cap > 0) BSQ_CHECK_PTR(y);
    BSQ_CHECK_PTR(dout);
  }
  BSQ_CHECK_PTR(pos);
  BSQ_CHECK_PTR(dweights);
  BSQ_DEVICE();
  return launch_combine_backward(T, H, cap, int(k), y, y_dtype == BSQ_BF16, pos, dout, dweights, as_stream(stream));
}

// ---------------------------------------------------------------- products --

bsq_status bsq_moe_matmul(int64_t T, int64_t cap, int64_t E, int64_t N, int64_t K, int64_t k, const uint8_t* a,
                          int a_dtype, const uint8_t* a_scales, const uint8_t* b, int b_dtype,
                          const uint8_t* b_scales, const int32_t* offsets, const int32_t* rows, void* out,
                          int out_dtype, void* stream) {
  BSQ_CHECK(T >= 0 && cap >= 0 && E >= 1 && N >= 0 && K >= 0 && k >= 1, BSQ_ERR_SHAPE,
            "negative size, or E or k below 1");
  BSQ_CHECK(known_dtype(a_dtype) && known_dtype(b_dtype) && known_dtype(out_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(is_fp8(a_dtype) && b_dtype == BSQ_E4M3, BSQ_ERR_UNSUPPORTED,
            "a must be E4M3 or E5M2 and b E4M3");
  BSQ_CHECK(is_wide(out_dtype), BSQ_ERR_UNSUPPORTED, "out_dtype must be F32 or BF16");
  BSQ_CHECK(K % 128 == 0 && N % 16 == 0, BSQ_ERR_UNSUPPORTED, "the library needs K % 128 == 0 and N % 16 == 0");
  BSQ_CHECK(E <= kMaxExperts, BSQ_ERR_UNSUPPORTED, "at most 1024 experts");
  BSQ_CHECK(T <= kMaxInt && cap <= kMaxRows && k <= kMaxInt && N <= (int64_t(1) << 30) && K <= kMaxContraction,
            BSQ_ERR_UNSUPPORTED, "extent too large");
  // the scale rows are addressed with 32-bit byte offsets
  BSQ_CHECK(elems_fit(E, N, K) && elems_fit(cap, N) && T * (K / 32) <= int64_t(0xFFFFFFFF) &&
                N * (K / 32) <= int64_t(0xFFFFFFFF),
            BSQ_ERR_UNSUPPORTED, "an operand too large");
  BSQ_CHECK((cap / 16 + E + 1) <= kMaxInt / ((N + 63) / 64 + 1), BSQ_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles");
  if (cap == 0 || N == 0) return ok();
  BSQ_CHECK_PTR(out);
  BSQ_CHECK_PTR(offsets);
  BSQ_CHECK(aligned16(rows), BSQ_ERR_ALIGN, "rows is not 16-byte aligned");
  if (K > 0 && T > 0) {
    BSQ_CHECK_PTR(a);
    BSQ_CHECK_PTR(b);
    BSQ_CHECK(a_scales != nullptr && b_scales != nullptr, BSQ_ERR_NULL, "scales are NULL");
    BSQ_CHECK(aligned4(a_scales) && aligned4(b_scales), BSQ_ERR_ALIGN, "scales must be 4-byte aligned");
  }
  BSQ_DEVICE();
  const MoeGemmLaunch L{T, cap, int(E), int(k), N, K, a, a_scales, b, b_scales, offsets, rows, out,
                        a_dtype == BSQ_E5M2, out_dtype == BSQ_BF16};
  return launch_moe_product(L, as_stream(stream));
}

bsq_status bsq_moe_wgrad(int64_t cap, int64_t E, int64_t N, int64_t K, const uint8_t* dyt, int dyt_dtype,
                         const uint8_t* dyt_scales, const uint8_t* xt, int xt_dtype, const uint8_t* xt_scales,
                         const int32_t* offsets, void* dW, int out_dtype, void* stream) {
  BSQ_CHECK(cap >= 0 && E >= 1 && N >= 0 && K >= 0, BSQ_ERR_SHAPE, "negative size, or E below 1");
  BSQ_CHECK(known_dtype(dyt_dtype) && known_dtype(xt_dtype) && known_dtype(out_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(is_fp8(dyt_dtype) && xt_dtype == BSQ_E4M3, BSQ_ERR_UNSUPPORTED,
            "dyt must be E4M3 or E5M2 and xt E4M3");
  BSQ_CHECK(is_wide(out_dtype), BSQ_ERR_UNSUPPORTED, "out_dtype must be F32 or BF16");
  BSQ_CHECK(cap % 128 == 0, BSQ_ERR_SHAPE, "cap must be a multiple of 128");
  BSQ_CHECK(N % 16 == 0 && K % 16 == 0, BSQ_ERR_UNSUPPORTED, "the library needs N % 16 == 0 and K % 16 == 0");
  BSQ_CHECK(E <= kMaxExperts, BSQ_ERR_UNSUPPORTED, "at most 1024 experts");
  BSQ_CHECK(cap <= kMaxInt && N <= (int64_t(1) << 30) && K <= (int64_t(1) << 30), BSQ_ERR_UNSUPPORTED,
            "extent too large");
  BSQ_CHECK(elems_fit(E, N, K) && N * (cap / 32) <= int64_t(0xFFFFFFFF) && K * (cap / 32) <= int64_t(0xFFFFFFFF),
            BSQ_ERR_UNSUPPORTED, "an operand too large");
  BSQ_CHECK(((N + 127) / 128) * ((K + 127) / 128) <= kMaxInt / E, BSQ_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles");
  if (N == 0 || K == 0) return ok();
  BSQ_CHECK_PTR(dW);
  BSQ_CHECK_PTR(offsets);
  if (cap > 0) {
    BSQ_CHECK_PTR(dyt);
    BSQ_CHECK_PTR(xt);
    BSQ_CHECK(dyt_scales != nullptr && xt_scales != nullptr, BSQ_ERR_NULL, "scales are NULL");
    BSQ_CHECK(aligned4(dyt_scales) && aligned4(xt_scales), BSQ_ERR_ALIGN, "scales must be 4-byte aligned");
  }
  BSQ_DEVICE();
  const MoeGemmLaunch L{0, cap, int(E), 1, N, K, dyt, dyt_scales, xt, xt_scales, offsets, nullptr, dW,
                        dyt_dtype == BSQ_E5M2, out_dtype == BSQ_BF16};
  return launch_moe_wgrad(L, as_stream(stream));
}

// -------------------------------------------------------------------- gate --

static bsq_status gate_check(int64_t R, int64_t F, int dtype, int code_dtype) {
  BSQ_CHECK(R >= 0 && F >= 0, BSQ_ERR_SHAPE, "negative size");
  BSQ_CHECK(elems_fit(R, F, 2), BSQ_ERR_UNSUPPORTED, "more than 2^60 elements");
  BSQ_CHECK(known_dtype(dtype) && known_dtype(code_dtype), BSQ_ERR_DTYPE, "unknown dtype");
  BSQ_CHECK(is_wide(dtype), BSQ_ERR_UNSUPPORTED, "values must be F32 or BF16");
  BSQ_CHECK(is_fp8(code_dtype), BSQ_ERR_UNSUPPORTED, "code_dtype must be E4M3 or E5M2");
  BSQ_CHECK(F % 32 == 0, BSQ_ERR_SHAPE, "F must be a multiple of 32");
  return BSQ_OK;
}

bsq_status bsq_swiglu_mx(int64_t R, int64_t F, const void* gu, int gu_dtype, int code_dtype, uint8_t* h,
                         uint8_t* h_scales, uint8_t* ht, uint8_t* ht_scales, uint8_t* kept, uint8_t* kept_scales,
                         void* stream) {
  const bsq_status s = gate_check(R, F, gu_dtype, code_dtype);
  if (s != BSQ_OK) return s;
  BSQ_CHECK(ht == nullptr || R % 32 == 0, BSQ_ERR_SHAPE, "R must be a multiple of 32 for the transposed codes");
  BSQ_CHECK((ht == nullptr) == (ht_scales == nullptr) && (kept == nullptr) == (kept_scales == nullptr), BSQ_ERR_NULL,
            "codes and their scales come together");
  BSQ_CHECK(R <= kMaxInt * 2048 / (F < 1 ? 1 : F), BSQ_ERR_UNSUPPORTED, "more than 2^31 - 1 workgroups");
  if (R == 0 || F == 0) return ok();
  BSQ_CHECK_PTR(gu);
  BSQ_CHECK_PTR(h);
  BSQ_CHECK(h_scales != nullptr, BSQ_ERR_NULL, "h_scales is NULL");
  BSQ_CHECK(aligned16(ht) && aligned16(kept), BSQ_ERR_ALIGN, "ht or kept is not 16-byte aligned");
  BSQ_DEVICE();
  return launch_swiglu_mx(R, F, gu, gu_dtype == BSQ_BF16, code_dtype == BSQ_E5M2, h, h_scales, ht, ht_scales, kept,
                          kept_scales, as_stream(stream));
}

bsq_status bsq_swiglu_mx_backward(int64_t R, int64_t F, const uint8_t* kept, int code_dtype,
                                  const uint8_t* kept_scales, const void* dh, int dh_dtype, void* dgu, void* stream) {
  const bsq_status s = gate_check(R, F, dh_dtype, code_dtype);
  if (s != BSQ_OK) return s;
  if (R == 0 || F == 0) return ok();
  BSQ_CHECK_PTR(kept);
  BSQ_CHECK(kept_scales != nullptr, BSQ_ERR_NULL, "kept_scales is NULL");
  BSQ_CHECK_PTR(dh);
  BSQ_CHECK_PTR(dgu);
  BSQ_DEVICE();
  return launch_swiglu_mx_backward(R, F, kept, kept_scales, code_dtype == BSQ_E5M2, dh, dh_dtype == BSQ_BF16, dgu,
                                   as_stream(stream));
}

}  // extern "C"
