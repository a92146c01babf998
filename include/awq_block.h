/*
 * awq_block.h - C ABI of the operators that stand around the W4A16 products of a decoder
 * block (awq.h) on MI355X (gfx950): the product with its element-wise tail, rotary
 * positions with the write into a paged cache, causal attention over packed prompts, and
 * attention of new or drafted tokens over the cache.
 *
 * Conventions are those of awq.h: status codes, device pointers aligned to 16 bytes, calls
 * asynchronous on `stream`, every argument checked before any launch, nothing allocated or
 * retained. In addition:
 *   - Index arrays (int32, int64, float32) need their elements' alignment only.
 *   - Elements are binary16 (AWQ_DT_F16) or bfloat16 (AWQ_DT_BF16); sums, softmax
 *     statistics and rotations are float32. Attention rounds probabilities to the element
 *     type before they meet v (the matrix instructions' operands), and divides by the sum of
 *     the rounded ones; outputs are rounded once.
 *   - Tokens are packed: x[token][head][d] with the head's D elements contiguous and the
 *     strides of the token and of the head (in elements) given, so that q, k and v may be
 *     views of one fused projection. Strides are multiples of 8 elements, a token's less
 *     than 2^23 (those of heads, and of a cache, are not limited); D is a multiple of 8,
 *     D <= 128. At most 4096 heads and 2^30 tokens.
 *   - `cu[B + 1]` (device, int32, not decreasing, cu[0] = 0) gives sequence b the packed
 *     tokens [cu[b], cu[b + 1]). Values are clamped to [0, tokens] on the device; outputs
 *     of tokens in no sequence are not written.
 *   - Query head h reads key / value head h / (Hq / Hkv).
 *   - Attention: what a row does not see never reaches it, infinities and NaN included. What it
 *     sees and is NaN makes the row NaN (a key) or that channel of it (a value); a visible
 *     infinity in a value gives infinity or, where its probability rounds to 0, NaN. Sums of
 *     finite values stay finite up to the type's largest; for that, bfloat16 values below
 *     about 2^-75 lose digits.
 *   - A paged cache holds position i of a sequence in slot i % page_size of page
 *     block_table[b][i / page_size]; a slot index is page * page_size + slot.
 */
#ifndef AWQ_BLOCK_H_
#define AWQ_BLOCK_H_

#include "awq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define AWQ_DT_F16 0
#define AWQ_DT_BF16 1

#define AWQ_ACT_NONE 0
#define AWQ_ACT_RELU 1
#define AWQ_ACT_GELU 2      /* v (1 + erf(v / sqrt 2)) / 2                          */
#define AWQ_ACT_GELU_TANH 3 /* v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2   */
#define AWQ_ACT_SILU 4      /* v / (1 + exp(-v))                                    */

/* What awq_gemm_fused does with a sum v of output n, row m; each pointer may be NULL. */
typedef struct awq_epilogue {
  const uint16_t* bias;     /* device, [N] binary16                                 */
  const uint16_t* mul;      /* device, [M][N] binary16 (a gated activation's factor) */
  const uint16_t* residual; /* device, [M][N] binary16                              */
  int32_t act;              /* AWQ_ACT_*                                            */
  int32_t reserved;         /* 0                                                    */
} awq_epilogue;

/*
 * awq_gemm_fused - awq_gemm with the element-wise tail of a decoder's projections:
 *   y[m][n] = binary16( act(v + bias[n]) * mul[m][n] + residual[m][n] ),
 * v the float32 sum that awq_gemm would round. Any M; the arguments, kernels, choice by
 * shape and workspace (awq_workspace_bytes) are awq_gemm's. mul and residual may be y
 * itself (each element is read by the thread that then writes it).
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE, HIP.
 */
int awq_gemm_fused(const uint16_t* x, const uint16_t* inv_s_c, const void* packed, int64_t M,
                   int64_t N, int64_t K, int32_t group, int32_t fmt, const awq_epilogue* epilogue,
                   uint16_t* y, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * awq_rope - rotary positions for q and k, and the write of k and v into a paged cache.
 * For pair i < rot_dim / 2 of a head, with angle = positions[t] * inv_freq[i]:
 *   out[a_i] = scale * (x[a_i] cos(angle) - x[b_i] sin(angle))
 *   out[b_i] = scale * (x[b_i] cos(angle) + x[a_i] sin(angle))
 * (a_i, b_i) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved != 0. inverse != 0
 * turns by -angle. Elements rot_dim .. D - 1 are copied. The angle is formed and reduced
 * in float64 (a position of 10^5 leaves no digits of it in float32).
 * q and k are rotated into q_out and k_out (either may be NULL; q_out may be q itself, k_out
 * k itself). With k_cache the rotated k, with v_cache v goes to slot slots[t] of the cache;
 * tokens whose slot is negative or past the cache are not stored.
 */
typedef struct awq_rope_args {
  const void* q; /* [tokens][q_heads][D], or NULL (then q_heads is ignored) */
  void* q_out;
  const void* k; /* [tokens][kv_heads][D], or NULL */
  void* k_out;   /* or NULL */
  const void* v; /* [tokens][kv_heads][D]; required with v_cache */
  void* k_cache; /* [pages][..], or NULL */
  void* v_cache; /* same shape and strides as k_cache, or NULL */
  const int32_t* positions; /* [tokens] */
  const float* inv_freq;    /* [rot_dim / 2] */
  const int64_t* slots;     /* [tokens]; required with a cache */
  int64_t tokens;
  int64_t q_token, q_head, qo_token, qo_head; /* strides */
  int64_t k_token, k_head, ko_token, ko_head, v_token, v_head;
  int64_t cache_page, cache_head, cache_slot;
  int64_t pages;
  int32_t page_size, q_heads, kv_heads, head_dim, rot_dim, dtype, interleaved, inverse;
  float scale;
  int32_t reserved; /* 0 */
} awq_rope_args;

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, HIP. tokens == 0 launches nothing. */
int awq_rope(const awq_rope_args* args, hipStream_t stream);

/*
 * awq_attn_prompt - causal attention of packed prompts:
 *   out[t][h] = sum over j <= t of t's sequence of p_j v_j,  p = softmax(scale q_t . k_j)
 * scale is finite and positive. (tokens / 128 + seqs) * q_heads <= 2^24 - 4096.
 */
typedef struct awq_attn_prompt_args {
  const void* q;   /* [tokens][q_heads][D] */
  const void* k;   /* [tokens][kv_heads][D] */
  const void* v;   /* [tokens][kv_heads][D] */
  void* out;       /* [tokens][q_heads][D], written */
  const int32_t* cu; /* [seqs + 1] */
  int64_t tokens, seqs;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head; /* strides */
  int32_t q_heads, kv_heads, head_dim, dtype;
  float scale;
  int32_t reserved; /* 0 */
} awq_attn_prompt_args;

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, HIP. tokens == 0 or seqs == 0 launches
 * nothing. */
int awq_attn_prompt(const awq_attn_prompt_args* args, hipStream_t stream);

/* Most tokens of one sequence in an awq_attn_tree call (one bit of a mask word each). */
#define AWQ_TREE_MAX_TOKENS 64

/*
 * awq_attn_tree - attention of the last tokens of each sequence over its paged cache.
 * Sequence b has ctx_lens[b] positions of context and T = cu_q[b + 1] - cu_q[b] new tokens
 * (at most max_q, at most AWQ_TREE_MAX_TOKENS) whose keys and values already stand in the
 * cache at positions ctx_lens[b] .. ctx_lens[b] + T - 1 (awq_rope puts them there). Token t
 * sees the whole context, and new token j where bit j of mask[cu_q[b] + t] is set (a tree of
 * drafted tokens: its ancestors and itself); without a mask, the new tokens j <= t. T == 1
 * is plain decoding. A token that sees nothing gets zeros. Slots past the sequence's end are
 * not seen.
 * block_table rows hold table_width entries; positions past table_width * page_size are
 * not there (the length is clamped), page numbers are clamped to [0, pages - 1].
 * scale is finite and positive. At most 65535 sequences, table_width * page_size < 2^30,
 * tokens * q_heads <= 2^25; with pages of a few positions and thousands of heads in a group,
 * less (UNSUPPORTED where row blocks times splits of the context exceed a launch).
 * ws: device, awq_attn_tree_workspace_bytes() bytes (the partial results of a context split
 * over workgroups; overwritten by every call), may be NULL with ws_bytes == 0 where that is 0.
 */
typedef struct awq_attn_tree_args {
  const void* q;       /* [tokens][q_heads][D] */
  const void* k_cache; /* [pages] x [kv_heads] x [page_size] x [D], strides below */
  const void* v_cache; /* same shape and strides */
  void* out;           /* [tokens][q_heads][D], written */
  const int32_t* block_table; /* [seqs][table_width] */
  const int32_t* ctx_lens;    /* [seqs] */
  const int32_t* cu_q;        /* [seqs + 1] */
  const uint64_t* mask;       /* [tokens], or NULL */
  void* ws;
  size_t ws_bytes;
  int64_t tokens, seqs, table_width, pages;
  int64_t q_token, q_head, o_token, o_head; /* strides */
  int64_t cache_page, cache_head, cache_slot;
  int32_t page_size, max_q, q_heads, kv_heads, head_dim, dtype;
  float scale;
  int32_t reserved; /* 0 */
} awq_attn_tree_args;

/* Workspace of an awq_attn_tree call; 0 where none is used, and for sizes it would refuse. */
size_t awq_attn_tree_workspace_bytes(int64_t tokens, int64_t seqs, int64_t table_width,
                                     int32_t page_size, int32_t max_q, int32_t q_heads,
                                     int32_t kv_heads, int32_t head_dim);

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE, HIP. tokens == 0 or seqs == 0
 * launches nothing. */
int awq_attn_tree(const awq_attn_tree_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_BLOCK_H_ */
