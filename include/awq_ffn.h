/*
 * awq_ffn.h - C ABI of the operators of a decoder's feed-forward half on MI355X (gfx950),
 * beside the W4A16 products (awq.h) and the operators around them (awq_block.h): the
 * root-mean-square norm with the residual's addition and an output in 8 bits, the product
 * in 8-bit integers that reads it, the router of a mixture of experts, and the layer of
 * W4A16 experts for a few tokens.
 *
 * Conventions are those of awq.h and awq_block.h: status codes, device pointers aligned to
 * 16 bytes (index and float32 arrays to their elements), calls asynchronous on `stream`,
 * every argument checked before any launch, nothing allocated or retained, elements binary16
 * (AWQ_DT_F16) or bfloat16 (AWQ_DT_BF16), outputs rounded once. Structures' `reserved` is 0.
 * Outputs must not overlap inputs except where an entry says so.
 */
#ifndef AWQ_FFN_H_
#define AWQ_FFN_H_

#include "awq_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * awq_rms_norm - for each token's row of `width` elements:
 *   h = x + residual, rounded to the element type (without a residual: h = x)
 *   v = h * weight / sqrt(mean(h^2) + eps)                            (float32)
 *   y = v rounded to the element type;  q = rint(v / s),  s = max|v| / 127
 * h_out, y and (q with scale) are each written where given; at least one of y and q is. h_out
 * may be x or residual, and y may be x or residual (the same address and stride).
 * Rows: strides of x, residual, h_out and y in elements, of q in bytes; at least width,
 * multiples of 8. width is a multiple of 8, 8 <= width <= 32768. eps is at least 1e-30.
 * Sums are float32; rows whose squares pass its range are summed scaled down.
 * 8-bit rows: s is formed as the float32 product of max|v| with float32's 1 / 127 (a unit in the
 * last place beside the quotient at times), and q from the quotient by that s. A row with no |v|
 * above 1e-30 gets scale 0 and codes 0; one that holds a v that is not finite gets scale NaN and
 * codes 0 (the row of a product with it is NaN).
 */
typedef struct awq_rms_norm_args {
  const void* x;        /* [tokens][width] */
  const void* residual; /* [tokens][width], or NULL */
  const void* weight;   /* [width], or NULL: ones */
  void* h_out;          /* [tokens][width], or NULL; needs residual */
  void* y;              /* [tokens][width], or NULL */
  int8_t* q;            /* [tokens][width], or NULL */
  float* scale;         /* [tokens]; required with q */
  int64_t tokens;
  int64_t x_stride, residual_stride, h_stride, y_stride, q_stride;
  int32_t width, dtype;
  float eps;
  int32_t reserved;
} awq_rms_norm_args;

/* Errors: INVALID_ARG, UNSUPPORTED (width or tokens too large), MISALIGNED, HIP. tokens == 0
 * launches nothing. At most 2^30 tokens. */
int awq_rms_norm(const awq_rms_norm_args* args, hipStream_t stream);

/*
 * awq_quant_i8 - 8-bit rows of x without a norm: v = x * inv_s_c (float32; inv_s_c of the
 * element type, NULL: ones), s = max|v| / 127, q = rint(v / s). Rows, limits and what is not
 * finite as in awq_rms_norm.
 */
typedef struct awq_quant_i8_args {
  const void* x;       /* [tokens][width] */
  const void* inv_s_c; /* [width], or NULL */
  int8_t* q;           /* [tokens][width] */
  float* scale;        /* [tokens] */
  int64_t tokens, x_stride, q_stride;
  int32_t width, dtype;
} awq_quant_i8_args;

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, HIP. tokens == 0 launches nothing. */
int awq_quant_i8(const awq_quant_i8_args* args, hipStream_t stream);

/* Bytes of the packed 8-bit layer of N outputs and K inputs (0 for sizes that are refused). */
size_t awq_packed_i8_bytes(int64_t N, int64_t K);

/*
 * awq_pack_i8 - a weight matrix w [N][K] (contiguous, `dtype`) in 8 bits with a scale for
 * each output channel: v = w * s_c (s_c [K] of the same type, NULL: ones; exact in float32),
 * s = max over k |v| / 127, q = rint(v / s). Rows of zeros and rows that are not finite as in
 * awq_rms_norm. Layout of `packed`, rows padded to Np = 16 ceil(N / 16) and channels to
 * Kp = 64 ceil(K / 64) with zeros:
 *   codes  at offset 0: unit (t, u), t < Np / 16, u < Kp / 64, at (t * Kp / 64 + u) * 1024;
 *          in a unit, bytes 16 l .. 16 l + 15 are row 16 t + l % 16, channels
 *          64 u + 16 (l / 16) .. + 15, l < 64;
 *   scales at offset Np * Kp: float32 [Np];
 *   the whole rounded up to 256 bytes.
 * N % 8 == 0, K % 16 == 0 (INVALID_ARG otherwise); K <= 131056 (the sums of products stay in
 * 32 bits), Np * Kp < 2^31 (UNSUPPORTED otherwise).
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE (packed_bytes too small), HIP.
 */
int awq_pack_i8(const void* w, const void* s_c, int64_t N, int64_t K, int32_t dtype, void* packed,
                size_t packed_bytes, hipStream_t stream);

/*
 * awq_gemm_i8 - product in 8-bit integers with a scale for each token and each channel:
 *   y[m][n] = act(scale[m] * s[n] * sum over k of q[m][k] w[n][k] + bias[n]) * mul[m][n]
 *             + residual[m][n]
 * The sum over k is exact (32-bit integers); the rest is float32, rounded once to `dtype`,
 * which is that of bias, mul and residual too. The product of the sum and both scales stays in
 * range where it is in range itself, for scales of channels below 2^104. act is AWQ_ACT_*.
 * Codes may be -128 .. 127. mul and residual may be y itself. q's rows are q_stride bytes apart (>= K, a multiple of
 * 16); y, mul and residual are contiguous. Limits of N and K are awq_pack_i8's; M < 2^30,
 * (M / 64 + 1) * (N / 16 + 1) <= 2^24 - 2^18.
 * ws: device, awq_gemm_i8_workspace_bytes() bytes, overwritten; may be NULL with ws_bytes == 0
 * where that is 0.
 */
typedef struct awq_gemm_i8_args {
  const int8_t* q;      /* [M][K] */
  const float* scale;   /* [M] */
  const void* packed;   /* awq_pack_i8's */
  const void* bias;     /* [N], or NULL */
  const void* mul;      /* [M][N], or NULL */
  const void* residual; /* [M][N], or NULL */
  void* y;              /* [M][N] */
  void* ws;
  size_t ws_bytes;
  int64_t M, N, K, q_stride;
  int32_t dtype, act;
} awq_gemm_i8_args;

/* Workspace of an awq_gemm_i8 call; 0 where none is used, and for sizes it would refuse. */
size_t awq_gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE, HIP. M == 0 launches nothing. */
int awq_gemm_i8(const awq_gemm_i8_args* args, hipStream_t stream);

#define AWQ_SCORE_SOFTMAX 0
#define AWQ_SCORE_SIGMOID 1

/*
 * awq_moe_route - which k of E experts each token takes, and with what weights.
 *   logit[e] = sum over c of x[t][c] w[e][c]      (float64: which expert is a border)
 *   p = softmax(logit) over all experts, or 1 / (1 + exp(-logit)) of each
 *   choice = logit (softmax) or p (sigmoid), + bias[e] where given
 *   ids[t] = the k largest choices, largest first, ties to the lowest index; a choice that is
 *            NaN stands behind all others
 *   weights[t][j] = scale * p[ids[t][j]], divided by their sum over j where renormalize != 0
 *            (0 where that sum is 0)
 * The bias is one for the choice alone, of logits or of sigmoids: not a linear router's bias,
 * which its weights would show too, and not one that is added to softmax's probabilities.
 * k <= E <= 1024, k <= 32, tokens <= 2^20, hidden a multiple of 8 up to 65536; x's rows x_stride
 * elements apart (a multiple of 8), w contiguous.
 * ws: device, awq_moe_route_workspace_bytes() bytes, overwritten; may be NULL with ws_bytes == 0
 * where that is 0 (a few tokens with a small router).
 */
typedef struct awq_moe_route_args {
  const void* x;     /* [tokens][hidden] */
  const void* w;     /* [E][hidden] */
  const float* bias; /* [E], or NULL */
  int32_t* ids;      /* [tokens][k] */
  float* weights;    /* [tokens][k] */
  void* ws;
  size_t ws_bytes;
  int64_t tokens, x_stride;
  int32_t hidden, experts, k, dtype, score, renormalize;
  float scale;
  int32_t reserved;
} awq_moe_route_args;

/* Workspace of an awq_moe_route call; 0 where none is used, and for sizes it would refuse. */
size_t awq_moe_route_workspace_bytes(int64_t tokens, int32_t hidden, int32_t experts);

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE, HIP. tokens == 0 launches nothing. */
int awq_moe_route(const awq_moe_route_args* args, hipStream_t stream);

/* Most tokens and most experts per token of an awq_moe call. */
#define AWQ_MOE_MAX_TOKENS 64
#define AWQ_MOE_MAX_K 32

/*
 * awq_moe - a layer of gated W4A16 experts for a few tokens:
 *   g = Wg[e] X', u = Wu[e] X', X' = binary16(x[t] * inv_in[e]),  e = ids[t][j]
 *   a = binary16(act(g) * u * inv_down[e])
 *   y[t] = residual[t] + sum over j of weights[t][j] * Wd[e] a
 * Sums are float32, in an order that the call's sizes and ids alone decide. Weights are the
 * packed layout of awq_repack, dequantized exactly (binary16((q - z) s)): gate and up [E]
 * layers of ffn outputs and hidden inputs, down [E] layers of hidden outputs and ffn inputs,
 * each stack's layers awq_repacked_bytes() apart. inv_in [E][hidden], or [hidden] for all
 * experts with inv_in_stride == 0; inv_down [E][ffn] or [ffn] likewise; binary16, NULL: ones.
 * An id outside [0, E) takes part in nothing (an expert of another device); a token may name
 * an expert twice. A token without an expert gets its residual, or zeros. y may be x or
 * residual (the same address and stride). Values of a past binary16 (65504) are infinities.
 * hidden and ffn are multiples of 128 (and of group), E <= 1024, tokens <= AWQ_MOE_MAX_TOKENS,
 * k <= AWQ_MOE_MAX_K. Rows of x, residual and y are strides (elements, multiples of 8) apart.
 * ws: device, awq_moe_workspace_bytes() bytes, overwritten.
 */
typedef struct awq_moe_args {
  const uint16_t* x;        /* [tokens][hidden] */
  const int32_t* ids;       /* [tokens][k] */
  const float* weights;     /* [tokens][k] */
  const void* gate;         /* [E] packed layers */
  const void* up;
  const void* down;
  const uint16_t* inv_in;   /* or NULL */
  const uint16_t* inv_down;  /* or NULL */
  const uint16_t* residual; /* [tokens][hidden], or NULL */
  uint16_t* y;              /* [tokens][hidden] */
  void* ws;
  size_t ws_bytes;
  int64_t tokens, x_stride, residual_stride, y_stride, inv_in_stride, inv_down_stride;
  int32_t hidden, ffn, experts, k, group, fmt, act;
  int32_t reserved;
} awq_moe_args;

/* Workspace of an awq_moe call; 0 for sizes it would refuse. */
size_t awq_moe_workspace_bytes(int64_t tokens, int32_t hidden, int32_t ffn, int32_t k);

/* Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE, HIP. tokens == 0 launches nothing. */
int awq_moe(const awq_moe_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_FFN_H_ */
