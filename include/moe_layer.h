/*
 * moe_layer.h -- C ABI of the operators between a decoder layer's attention
 * (moe_kv4.h) and its experts (moe_int4.h), for one NVIDIA GB300 (sm_103a): the
 * residual's addition with the root-mean-square norm, matrix products with an
 * epilogue, and the routing to experts.  The conventions of moe_int4.h hold
 * (device pointers of the caller, stream-ordered asynchronous calls, MOE_OK or a
 * negative MOE_ERR_* code, no allocation); the entry points live in the same
 * library and moe_int4_strerror names their codes.  None needs a workspace.
 *
 * Matrices are rows of contiguous elements; a *_stride is the number of elements
 * from one row to the next (at least the row's length; with one row it is not used).
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  The first two are MOE_OUT_BF16 and MOE_OUT_F32. */
#define MOE_T_BF16 0
#define MOE_T_F32 1
#define MOE_T_F16 2
#define MOE_T_E4M3 3 /* 8 bits: sign, 4-bit exponent with bias 7, 3-bit mantissa, up to 448 */

/* Activations of moe_linear. */
#define MOE_ACT_NONE 0
#define MOE_ACT_RELU 1 /* max(y, 0); NaN stays NaN */
#define MOE_ACT_SILU 2 /* y / (1 + e^-y); 0 below -88.7, where e^-y leaves fp32 */
#define MOE_ACT_GELU 3 /* y (1 + erf(y / sqrt 2)) / 2, within 2^-23 |y| where 1 + erf cancels */

/* Kernels of moe_linear. */
#define MOE_LINEAR_SPLIT 1          /* a tile a cluster, whose blocks share the sum */
#define MOE_LINEAR_PAIRS_128 2      /* tiles of 256 x 128 on two SMs */
#define MOE_LINEAR_PAIRS_128_SUMS 3 /* the same, with the sum in parts */
#define MOE_LINEAR_PAIRS_256 4      /* tiles of 256 x 256 on two SMs */

/* Scores of moe_route_experts. */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

/*
 * moe_add_norm: the residual's addition and the root-mean-square norm of each row.
 *   h = x + residual                       rounded to the residual's type
 *   y = h * (1 / sqrt(mean(h^2) + eps)) * weight
 * In:  x         [rows][hidden], x_type MOE_T_BF16, _F32 or _F16
 *      residual  [rows][hidden] of residual_type (those three); NULL: h = x, and
 *                residual_out must be NULL
 *      weight    [hidden] of weight_type (those three); NULL: 1
 * Out: residual_out  h, of residual_type (may be residual itself; NULL: not kept)
 *      out       y, of out_type (those three); may be x itself where type and stride
 *                are the same; NULL: not wanted
 *      codes     e4m3 codes of y / scale, nearest even, with one scale for each row:
 *                scales[row] = max(max|y| / 448, 2^-100); both NULL: not wanted
 * Everything is fp32 with each operation rounded on its own.  The sum of squares is
 * held in two fp32 numbers (some 45 bits) and rounded to one at the end, so that the order
 * of its parts shows in about one row of a million, whose sum lies next to a rounding: total * fp32(1/hidden), + eps, square root, reciprocal,
 * h * that, * weight; for the codes y * (1 / scale) with scale = max|y| * fp32(1/448).
 * Rows whose sum leaves fp32 (values beyond 1e18, or tiny ones with eps = 0) are added
 * up in 64 bits, and where 1 / sqrt leaves it too, multiplied by a power of two first.  A
 * row of zeros with eps = 0 becomes NaN (0 / 0).  A row that holds NaN becomes NaN; one
 * that holds an infinity (and no NaN) becomes 0, and NaN where the infinity was.  max|y|
 * does not count NaN.
 * Sizes: 0 <= rows <= 1<<20, 1 <= hidden <= 32768, 0 <= eps (finite).  Pointers need
 * their type's alignment only; rows that all begin at multiples of 16 bytes are
 * faster.  Errors: MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_ALIGN, MOE_ERR_UNSUPPORTED,
 * MOE_ERR_CUDA.
 */
int moe_add_norm(const void *x, int x_type, int64_t x_stride, const void *residual,
                 int residual_type, int64_t residual_stride, const void *weight, int weight_type,
                 float eps, int rows, int hidden, void *residual_out,
                 int64_t residual_out_stride, void *out, int out_type, int64_t out_stride,
                 uint8_t *codes, int64_t codes_stride, float *scales, moe_stream_t stream);

/*
 * moe_linear: a matrix product with its epilogue,
 *   out[m][n] = activation(sum_k x[m][k] w[n][k] * x_scale[m] * w_scale[n] + bias[n])
 *               * gate[m][n] + residual[m][n]
 * In:  x         [M][K], w [N][K], both of `type`: MOE_T_BF16, _F16 or _E4M3
 *      x_scale   fp32 [M], w_scale fp32 [N]; NULL: 1
 *      bias      fp32 [N]; NULL: 0
 *      gate      [M][N] of gate_type (MOE_T_BF16, _F32 or _F16); NULL: 1
 *      residual  [M][N] of residual_type (those three); NULL: 0
 * Out: out       [M][N] of out_type (those three); may be gate or residual itself
 *                where type and stride are the same, must not overlap x or w
 * Products are added up in fp32 by the tensor cores, the epilogue is fp32, and the
 * result is rounded once.  Where the result stays fp32 (or K is beyond 32 768 two-byte
 * elements) long sums are made of parts of 768 elements (1536 codes), since the tensor
 * cores cut a sum's last place again and again.  The order of the sum depends on the
 * sizes, types and alignments only, so the same call gives the same bits.
 * x and w: rows begin at multiples of 16 bytes (pointers 16-byte aligned, strides
 * multiples of 16 bytes); K itself may be any number.  The others need their type's
 * alignment only.  err: device uint32 or NULL; MOE_DEVERR_TIMEOUT is set where a wait
 * inside the kernel ran out (a bug guard; the output is then not valid).
 * Sizes: 0 <= M <= 1<<20, 1 <= N <= 1<<20, 1 <= K <= 1<<20; M == 0 is a no-op.
 * Errors: as moe_add_norm.
 */
int moe_linear(const void *x, int64_t x_stride, const float *x_scale, const void *w,
               int64_t w_stride, const float *w_scale, int type, const float *bias,
               int activation, const void *gate, int gate_type, int64_t gate_stride,
               const void *residual, int residual_type, int64_t residual_stride, void *out,
               int out_type, int64_t out_stride, int M, int N, int K, uint32_t *err,
               moe_stream_t stream);

/* The kernel that this thread's last moe_linear launched (sizes, types and alignments decide);
 * 0: none yet. */
int moe_linear_last_kernel(void);

/*
 * moe_route_experts: the experts of each token and their weights.
 *   s = sigmoid(logit), or the softmax of the token's logits     (scoring)
 *   c = s + bias                                                 what chooses
 * Experts form `groups` runs of E / groups.  The top_groups best groups are chosen by
 * their best c (group_best 1) or the sum of their two best (2), then the top_k experts
 * by c among the chosen groups' ones.  Groups and experts that are equal are taken in
 * ascending index.
 *   weight = s, divided by the sum of the chosen ones (renormalize), * scale
 * In:  logits    [M][E], type MOE_T_F32, _BF16 or _F16
 *      bias      fp32 [E]; NULL: 0
 * Out: topk_ids int32 [M][top_k], best first; topk_weights fp32 [M][top_k].
 * c is compared in 64 bits (where fp32 decides, by fp32), so the choice does not depend
 * on how an exponential was rounded; without a bias scores order as the logits do, and
 * experts, and groups by their best, are compared by these.  Renormalised weights are
 * formed relative to the largest chosen score and do not underflow together.
 * Masked experts: one whose logit is -inf or NaN, or whose bias is, is not available.
 * It is chosen after all available ones of the chosen groups, lower index first, with
 * weight 0; groups rank by their available experts (a sum by the one that is left), those
 * without any last.  +inf counts as the largest finite number.  So ids are always
 * distinct and inside [0, E).
 * Sizes: 0 <= M <= 1<<20, 1 <= E <= 1024, groups <= 32 and a divisor of E,
 * 1 <= top_groups <= groups, 1 <= top_k <= min(32, E / groups * top_groups); scale
 * finite.  Errors: as moe_add_norm.
 */
int moe_route_experts(const void *logits, int type, int64_t stride, const float *bias, int M,
                      int E, int top_k, int scoring, int groups, int top_groups, int group_best,
                      int renormalize, float scale, int32_t *topk_ids, float *topk_weights,
                      moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
