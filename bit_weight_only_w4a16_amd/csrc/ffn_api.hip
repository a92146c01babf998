// C ABI entry points of the feed-forward operators (awq_ffn.h): argument checks (all before
// any launch), then the launchers.
#include "ffn_internal.hpp"

#include <math.h>

namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 30, kMaxStride = int64_t{1} << 23;
constexpr int kMaxWidth = 32768, kMaxHidden = 65536, kMaxExperts = 1024;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

#define AWQ_TRY(expr)              \
  do {                             \
    const int rc_ = (expr);        \
    if (rc_ != AWQ_OK) return rc_; \
  } while (0)

int check_rows(int64_t tokens, int32_t width, int32_t dtype) {
  if (tokens < 0 || width <= 0 || width % 8 != 0) return AWQ_ERR_INVALID_ARG;
  if (dtype != AWQ_DT_F16 && dtype != AWQ_DT_BF16) return AWQ_ERR_INVALID_ARG;
  if (width > kMaxWidth || tokens > kMaxTokens) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}
int check_stride(const void* p, int64_t stride, int32_t width) {
  if (p == nullptr) return AWQ_OK;
  if (stride < width) return AWQ_ERR_INVALID_ARG;
  if (stride % 8 != 0 || !aligned16(p)) return AWQ_ERR_MISALIGNED;
  return stride < (int64_t{1} << 31) ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}

int check_i8_shape(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0 || N % 8 != 0 || K % 16 != 0) return AWQ_ERR_INVALID_ARG;
  if (K > 131056 || N >= (int64_t{1} << 31)) return AWQ_ERR_UNSUPPORTED;
  const awq::I8Layout l = awq::make_i8_layout(N, K);
  return l.scales_off < (int64_t{1} << 31) ? AWQ_OK : AWQ_ERR_UNSUPPORTED;
}
int check_i8_product(int64_t M, int64_t N, int64_t K) {
  AWQ_TRY(check_i8_shape(N, K));
  if (M < 0) return AWQ_ERR_INVALID_ARG;
  if (M >= kMaxTokens || (M / 64 + 1) * (N / 16 + 1) > (int64_t{1} << 24) - (1 << 18)) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

int check_route_sizes(int64_t tokens, int32_t hidden, int32_t experts) {
  if (tokens < 0 || hidden <= 0 || hidden % 8 != 0 || experts <= 0) return AWQ_ERR_INVALID_ARG;
  if (tokens > (int64_t{1} << 20) || hidden > kMaxHidden || experts > kMaxExperts) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

int check_moe_sizes(int64_t tokens, int32_t hidden, int32_t ffn, int32_t k) {
  if (tokens < 0 || hidden <= 0 || ffn <= 0 || k <= 0) return AWQ_ERR_INVALID_ARG;
  if (tokens > AWQ_MOE_MAX_TOKENS || k > AWQ_MOE_MAX_K) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

}  // namespace

extern "C" {

int awq_rms_norm(const awq_rms_norm_args* a, hipStream_t stream) {
  if (a == nullptr || a->reserved != 0) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_rows(a->tokens, a->width, a->dtype));
  if (!isfinite(a->eps) || !(a->eps >= 1e-30f)) return AWQ_ERR_INVALID_ARG;
  if (a->tokens == 0) return AWQ_OK;
  if (a->x == nullptr || (a->y == nullptr && a->q == nullptr)) return AWQ_ERR_INVALID_ARG;
  if ((a->q != nullptr) != (a->scale != nullptr) || (a->h_out != nullptr && a->residual == nullptr))
    return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_stride(a->x, a->x_stride, a->width));
  AWQ_TRY(check_stride(a->residual, a->residual_stride, a->width));
  AWQ_TRY(check_stride(a->h_out, a->h_stride, a->width));
  AWQ_TRY(check_stride(a->y, a->y_stride, a->width));
  AWQ_TRY(check_stride(a->q, a->q_stride, a->width));
  if (!aligned16(a->weight) || !aligned4(a->scale)) return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_rms_norm(*a, stream));
}

int awq_quant_i8(const awq_quant_i8_args* a, hipStream_t stream) {
  if (a == nullptr) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_rows(a->tokens, a->width, a->dtype));
  if (a->tokens == 0) return AWQ_OK;
  if (a->x == nullptr || a->q == nullptr || a->scale == nullptr) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_stride(a->x, a->x_stride, a->width));
  AWQ_TRY(check_stride(a->q, a->q_stride, a->width));
  if (!aligned16(a->inv_s_c) || !aligned4(a->scale)) return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_quant_i8(*a, stream));
}

size_t awq_packed_i8_bytes(int64_t N, int64_t K) {
  if (check_i8_shape(N, K) != AWQ_OK) return 0;
  return static_cast<size_t>(awq::make_i8_layout(N, K).total_bytes);
}

int awq_pack_i8(const void* w, const void* s_c, int64_t N, int64_t K, int32_t dtype, void* packed,
                size_t packed_bytes, hipStream_t stream) {
  AWQ_TRY(check_i8_shape(N, K));
  if (dtype != AWQ_DT_F16 && dtype != AWQ_DT_BF16) return AWQ_ERR_INVALID_ARG;
  if (w == nullptr || packed == nullptr) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(s_c) || !aligned16(packed)) return AWQ_ERR_MISALIGNED;
  if (packed_bytes < awq_packed_i8_bytes(N, K)) return AWQ_ERR_WORKSPACE;
  return hip_status(awq::launch_pack_i8(w, s_c, N, K, dtype, packed, stream));
}

size_t awq_gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || check_i8_product(M, N, K) != AWQ_OK) return 0;
  return awq::gemm_i8_workspace_bytes(M, N, K);
}

int awq_gemm_i8(const awq_gemm_i8_args* a, hipStream_t stream) {
  if (a == nullptr) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_i8_product(a->M, a->N, a->K));
  if (a->dtype != AWQ_DT_F16 && a->dtype != AWQ_DT_BF16) return AWQ_ERR_INVALID_ARG;
  if (a->act < AWQ_ACT_NONE || a->act > AWQ_ACT_SILU) return AWQ_ERR_INVALID_ARG;
  if (a->ws == nullptr && a->ws_bytes != 0) return AWQ_ERR_INVALID_ARG;
  if (a->M == 0) return AWQ_OK;
  if (a->q == nullptr || a->scale == nullptr || a->packed == nullptr || a->y == nullptr) return AWQ_ERR_INVALID_ARG;
  if (a->q_stride < a->K) return AWQ_ERR_INVALID_ARG;
  if (a->q_stride % 16 != 0 || !aligned16(a->q) || !aligned4(a->scale) || !aligned16(a->packed) ||
      !aligned16(a->bias) || !aligned16(a->mul) || !aligned16(a->residual) || !aligned16(a->y) || !aligned16(a->ws))
    return AWQ_ERR_MISALIGNED;
  if (a->q_stride >= kMaxStride) return AWQ_ERR_UNSUPPORTED;
  if (a->ws_bytes < awq::gemm_i8_workspace_bytes(a->M, a->N, a->K)) return AWQ_ERR_WORKSPACE;
  return hip_status(awq::launch_gemm_i8(*a, stream));
}

size_t awq_moe_route_workspace_bytes(int64_t tokens, int32_t hidden, int32_t experts) {
  if (tokens == 0 || check_route_sizes(tokens, hidden, experts) != AWQ_OK) return 0;
  return awq::moe_route_workspace_bytes(tokens, hidden, experts);
}

int awq_moe_route(const awq_moe_route_args* a, hipStream_t stream) {
  if (a == nullptr || a->reserved != 0) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_route_sizes(a->tokens, a->hidden, a->experts));
  if (a->dtype != AWQ_DT_F16 && a->dtype != AWQ_DT_BF16) return AWQ_ERR_INVALID_ARG;
  if (a->score != AWQ_SCORE_SOFTMAX && a->score != AWQ_SCORE_SIGMOID) return AWQ_ERR_INVALID_ARG;
  if (a->k <= 0 || a->k > a->experts || !isfinite(a->scale)) return AWQ_ERR_INVALID_ARG;
  if (a->k > AWQ_MOE_MAX_K) return AWQ_ERR_UNSUPPORTED;
  if (a->ws == nullptr && a->ws_bytes != 0) return AWQ_ERR_INVALID_ARG;
  if (a->tokens == 0) return AWQ_OK;
  if (a->x == nullptr || a->w == nullptr || a->ids == nullptr || a->weights == nullptr) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_stride(a->x, a->x_stride, a->hidden));
  if (!aligned16(a->w) || !aligned4(a->bias) || !aligned4(a->ids) || !aligned4(a->weights) || !aligned16(a->ws))
    return AWQ_ERR_MISALIGNED;
  if (a->ws_bytes < awq::moe_route_workspace_bytes(a->tokens, a->hidden, a->experts)) return AWQ_ERR_WORKSPACE;
  return hip_status(awq::launch_moe_route(*a, stream));
}

size_t awq_moe_workspace_bytes(int64_t tokens, int32_t hidden, int32_t ffn, int32_t k) {
  if (tokens == 0 || check_moe_sizes(tokens, hidden, ffn, k) != AWQ_OK) return 0;
  // the limits of a layer that hold for all groups and formats, both ways round
  if (hidden % 128 != 0 || ffn % 128 != 0 || awq_repacked_bytes(ffn, hidden, 128, AWQ_FMT_SYM8) == 0 ||
      awq_repacked_bytes(hidden, ffn, 128, AWQ_FMT_SYM8) == 0)
    return 0;
  return awq::moe_workspace_bytes(tokens, hidden, ffn, k);
}

int awq_moe(const awq_moe_args* a, hipStream_t stream) {
  if (a == nullptr || a->reserved != 0) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_moe_sizes(a->tokens, a->hidden, a->ffn, a->k));
  if (a->experts <= 0 || a->group <= 0 || a->act < AWQ_ACT_NONE || a->act > AWQ_ACT_SILU) return AWQ_ERR_INVALID_ARG;
  if (a->fmt != AWQ_FMT_ASYM && a->fmt != AWQ_FMT_SYM8) return AWQ_ERR_INVALID_ARG;
  if (a->hidden % a->group != 0 || a->ffn % a->group != 0) return AWQ_ERR_INVALID_ARG;
  if (a->hidden % 128 != 0 || a->ffn % 128 != 0 || a->experts > kMaxExperts) return AWQ_ERR_UNSUPPORTED;
  // the limits of a layer, both ways round
  if (awq_repacked_bytes(a->ffn, a->hidden, a->group, a->fmt) == 0 ||
      awq_repacked_bytes(a->hidden, a->ffn, a->group, a->fmt) == 0)
    return AWQ_ERR_UNSUPPORTED;
  if (a->ws == nullptr && a->ws_bytes != 0) return AWQ_ERR_INVALID_ARG;
  if (a->tokens == 0) return AWQ_OK;
  if (a->x == nullptr || a->ids == nullptr || a->weights == nullptr || a->gate == nullptr || a->up == nullptr ||
      a->down == nullptr || a->y == nullptr)
    return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_stride(a->x, a->x_stride, a->hidden));
  AWQ_TRY(check_stride(a->residual, a->residual_stride, a->hidden));
  AWQ_TRY(check_stride(a->y, a->y_stride, a->hidden));
  if (a->inv_in != nullptr && a->inv_in_stride != 0) AWQ_TRY(check_stride(a->inv_in, a->inv_in_stride, a->hidden));
  if (a->inv_down != nullptr && a->inv_down_stride != 0) AWQ_TRY(check_stride(a->inv_down, a->inv_down_stride, a->ffn));
  if (!aligned4(a->ids) || !aligned4(a->weights) || !aligned16(a->gate) || !aligned16(a->up) || !aligned16(a->down) ||
      !aligned16(a->inv_in) || !aligned16(a->inv_down) || !aligned16(a->ws))
    return AWQ_ERR_MISALIGNED;
  if (a->ws_bytes < awq::moe_workspace_bytes(a->tokens, a->hidden, a->ffn, a->k)) return AWQ_ERR_WORKSPACE;
  return hip_status(awq::launch_moe(*a, stream));
}

}  // extern "C"
