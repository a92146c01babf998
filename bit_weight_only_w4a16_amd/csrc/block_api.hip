// C ABI entry points of the decoder-block operators (awq_block.h): argument checks (all
// before any launch), then the launchers.
#include "block_internal.hpp"
#include "epilogue.hpp"

#include <math.h>

namespace {

constexpr int64_t kMaxStride = int64_t{1} << 23;  // elements: 128 rows stay below 2^31 bytes
constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 4096, kMaxRows = int64_t{1} << 25;
constexpr int64_t kMaxBlocks = (int64_t{1} << 24) - 1;
constexpr int kMaxHeadDim = 128, kMaxHeads = 4096;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// index arrays: their elements' own alignment
inline bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

// heads and head size shared by the three operators
int check_heads(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype) {
  if (q_heads <= 0 || kv_heads <= 0 || head_dim <= 0) return AWQ_ERR_INVALID_ARG;
  if (dtype != AWQ_DT_F16 && dtype != AWQ_DT_BF16) return AWQ_ERR_INVALID_ARG;
  if (head_dim % 8 != 0) return AWQ_ERR_INVALID_ARG;
  if (head_dim > kMaxHeadDim || q_heads > kMaxHeads || kv_heads > kMaxHeads) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

// a packed operand: strides that hold a head's elements (one head may have any stride) and
// keep 16-byte accesses aligned
int check_strides(int64_t token, int64_t head, int32_t heads, int32_t head_dim) {
  if (token < 0 || head < 0) return AWQ_ERR_INVALID_ARG;
  if ((heads > 1 && head < head_dim) || token < head_dim) return AWQ_ERR_INVALID_ARG;
  if (token % 8 != 0 || head % 8 != 0) return AWQ_ERR_MISALIGNED;
  if (token >= kMaxStride) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

int check_cache(int64_t page, int64_t head, int64_t slot, int64_t pages, int32_t page_size, int32_t head_dim) {
  if (pages <= 0 || page_size <= 0) return AWQ_ERR_INVALID_ARG;
  if (page < 0 || head < 0 || slot < head_dim) return AWQ_ERR_INVALID_ARG;
  if (page % 8 != 0 || head % 8 != 0 || slot % 8 != 0) return AWQ_ERR_MISALIGNED;
  if (pages >= (int64_t{1} << 31)) return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

#define AWQ_TRY(expr)                 \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != AWQ_OK) return rc_;    \
  } while (0)

}  // namespace

extern "C" {

int awq_gemm_fused(const uint16_t* x, const uint16_t* inv_s_c, const void* packed, int64_t M, int64_t N,
                   int64_t K, int32_t group, int32_t fmt, const awq_epilogue* epilogue, uint16_t* y,
                   void* ws, size_t ws_bytes, hipStream_t stream) {
  AWQ_TRY(awq::check_product(x, inv_s_c, packed, M, N, K, group, fmt, y, ws, ws_bytes));
  if (epilogue == nullptr || epilogue->reserved != 0) return AWQ_ERR_INVALID_ARG;
  if (epilogue->act < AWQ_ACT_NONE || epilogue->act > AWQ_ACT_SILU) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(epilogue->bias) || !aligned16(epilogue->mul) || !aligned16(epilogue->residual))
    return AWQ_ERR_MISALIGNED;
  if (M == 0) return AWQ_OK;
  const awq::Epilogue e = {epilogue->bias, epilogue->mul, epilogue->residual, epilogue->act};
  return hip_status(
      awq::launch_gemm_fused(x, inv_s_c, packed, M, N, K, group, fmt, e, y, ws, ws_bytes, stream));
}

int awq_rope(const awq_rope_args* a, hipStream_t stream) {
  if (a == nullptr || a->reserved != 0 || a->tokens < 0) return AWQ_ERR_INVALID_ARG;
  if (a->tokens == 0) return AWQ_OK;
  if (a->q == nullptr && a->k == nullptr) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_heads(a->q != nullptr ? a->q_heads : 1, a->k != nullptr ? a->kv_heads : 1, a->head_dim,
                      a->dtype));
  if (a->rot_dim < 0 || a->rot_dim % 2 != 0 || a->rot_dim > a->head_dim)
    return AWQ_ERR_INVALID_ARG;
  if (!isfinite(a->scale)) return AWQ_ERR_INVALID_ARG;
  const bool cache = a->k_cache != nullptr || a->v_cache != nullptr;
  if ((a->q != nullptr) != (a->q_out != nullptr)) return AWQ_ERR_INVALID_ARG;
  if (a->k == nullptr && (a->k_out != nullptr || cache)) return AWQ_ERR_INVALID_ARG;
  if (a->k != nullptr && a->k_out == nullptr && a->k_cache == nullptr) return AWQ_ERR_INVALID_ARG;
  if (a->v_cache != nullptr && a->v == nullptr) return AWQ_ERR_INVALID_ARG;
  if (cache && a->slots == nullptr) return AWQ_ERR_INVALID_ARG;
  if (a->positions == nullptr || (a->rot_dim > 0 && a->inv_freq == nullptr)) return AWQ_ERR_INVALID_ARG;
  if (a->q != nullptr) {
    AWQ_TRY(check_strides(a->q_token, a->q_head, a->q_heads, a->head_dim));
    AWQ_TRY(check_strides(a->qo_token, a->qo_head, a->q_heads, a->head_dim));
  }
  if (a->k != nullptr) AWQ_TRY(check_strides(a->k_token, a->k_head, a->kv_heads, a->head_dim));
  if (a->k_out != nullptr) AWQ_TRY(check_strides(a->ko_token, a->ko_head, a->kv_heads, a->head_dim));
  if (a->v_cache != nullptr) AWQ_TRY(check_strides(a->v_token, a->v_head, a->kv_heads, a->head_dim));
  if (cache)
    AWQ_TRY(check_cache(a->cache_page, a->cache_head, a->cache_slot, a->pages, a->page_size, a->head_dim));
  if (!aligned16(a->q) || !aligned16(a->q_out) || !aligned16(a->k) || !aligned16(a->k_out) ||
      !aligned16(a->v) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned(a->positions, 4) ||
      !aligned(a->inv_freq, 4) || !aligned(a->slots, 8))
    return AWQ_ERR_MISALIGNED;
  if (a->tokens > kMaxTokens) return AWQ_ERR_UNSUPPORTED;
  return hip_status(awq::launch_rope(*a, stream));
}

int awq_attn_prompt(const awq_attn_prompt_args* a, hipStream_t stream) {
  if (a == nullptr || a->reserved != 0) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_heads(a->q_heads, a->kv_heads, a->head_dim, a->dtype));
  if (a->tokens < 0 || a->seqs < 0 || a->q_heads % a->kv_heads != 0) return AWQ_ERR_INVALID_ARG;
  if (!isfinite(a->scale) || !(a->scale > 0.0f)) return AWQ_ERR_INVALID_ARG;
  if (a->tokens == 0 || a->seqs == 0) return AWQ_OK;
  if (a->q == nullptr || a->k == nullptr || a->v == nullptr || a->out == nullptr || a->cu == nullptr)
    return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_strides(a->q_token, a->q_head, a->q_heads, a->head_dim));
  AWQ_TRY(check_strides(a->k_token, a->k_head, a->kv_heads, a->head_dim));
  AWQ_TRY(check_strides(a->v_token, a->v_head, a->kv_heads, a->head_dim));
  AWQ_TRY(check_strides(a->o_token, a->o_head, a->q_heads, a->head_dim));
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out) || !aligned(a->cu, 4))
    return AWQ_ERR_MISALIGNED;
  if (a->tokens > kMaxTokens || a->seqs > kMaxTokens) return AWQ_ERR_UNSUPPORTED;
  // workgroups of 128 query rows: a launch holds 2^32 threads
  if ((a->tokens / 128 + a->seqs) * a->q_heads > kMaxGroups)
    return AWQ_ERR_UNSUPPORTED;
  return hip_status(awq::launch_attn_prompt(*a, stream));
}

static int check_tree_sizes(int64_t tokens, int64_t seqs, int64_t table_width, int32_t page_size,
                            int32_t max_q, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  AWQ_TRY(check_heads(q_heads, kv_heads, head_dim, AWQ_DT_F16));
  if (tokens < 0 || seqs < 0 || table_width <= 0 || page_size <= 0 || max_q <= 0 || q_heads % kv_heads != 0)
    return AWQ_ERR_INVALID_ARG;
  if (max_q > AWQ_TREE_MAX_TOKENS || seqs > 65535 || tokens > kMaxTokens) return AWQ_ERR_UNSUPPORTED;
  if (table_width >= (int64_t{1} << 31) || table_width * page_size >= (int64_t{1} << 30))
    return AWQ_ERR_UNSUPPORTED;
  // a wavefront per row in the second launch, which holds 2^32 threads; with at most 2^21
  // splits (pages of one position) of 130 floats a row the workspace's size fits 64 bits
  if (tokens * q_heads > kMaxRows) return AWQ_ERR_UNSUPPORTED;
  // workgroups of 256 threads along x, of which a launch holds 2^32
  if (awq::attn_tree_blocks(seqs, table_width, page_size, max_q, q_heads, kv_heads, head_dim) > kMaxBlocks)
    return AWQ_ERR_UNSUPPORTED;
  return AWQ_OK;
}

size_t awq_attn_tree_workspace_bytes(int64_t tokens, int64_t seqs, int64_t table_width, int32_t page_size,
                                     int32_t max_q, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (tokens == 0 || seqs == 0) return 0;
  if (check_tree_sizes(tokens, seqs, table_width, page_size, max_q, q_heads, kv_heads, head_dim) != AWQ_OK)
    return 0;
  return awq::attn_tree_workspace_bytes(tokens, seqs, table_width, page_size, max_q, q_heads, kv_heads,
                                        head_dim);
}

int awq_attn_tree(const awq_attn_tree_args* a, hipStream_t stream) {
  if (a == nullptr || a->reserved != 0) return AWQ_ERR_INVALID_ARG;
  if (a->dtype != AWQ_DT_F16 && a->dtype != AWQ_DT_BF16) return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_tree_sizes(a->tokens, a->seqs, a->table_width, a->page_size, a->max_q, a->q_heads,
                           a->kv_heads, a->head_dim));
  if (!isfinite(a->scale) || !(a->scale > 0.0f)) return AWQ_ERR_INVALID_ARG;
  if (a->ws == nullptr && a->ws_bytes != 0) return AWQ_ERR_INVALID_ARG;
  if (a->tokens == 0 || a->seqs == 0) return AWQ_OK;
  if (a->q == nullptr || a->k_cache == nullptr || a->v_cache == nullptr || a->out == nullptr ||
      a->block_table == nullptr || a->ctx_lens == nullptr || a->cu_q == nullptr)
    return AWQ_ERR_INVALID_ARG;
  AWQ_TRY(check_strides(a->q_token, a->q_head, a->q_heads, a->head_dim));
  AWQ_TRY(check_strides(a->o_token, a->o_head, a->q_heads, a->head_dim));
  AWQ_TRY(check_cache(a->cache_page, a->cache_head, a->cache_slot, a->pages, a->page_size, a->head_dim));
  if (!aligned16(a->q) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->out) ||
      !aligned(a->block_table, 4) || !aligned(a->ctx_lens, 4) || !aligned(a->cu_q, 4) ||
      !aligned(a->mask, 8) || !aligned16(a->ws))
    return AWQ_ERR_MISALIGNED;
  if (a->ws_bytes < awq::attn_tree_workspace_bytes(a->tokens, a->seqs, a->table_width, a->page_size, a->max_q,
                                                   a->q_heads, a->kv_heads, a->head_dim))
    return AWQ_ERR_WORKSPACE;
  return hip_status(awq::launch_attn_tree(*a, stream));
}

}  // extern "C"
