/*
 * sparse-moe-4bit for GB300 (sm_103a): C ABI of what a decode step has between
 * and behind the layers of moe.h, gdn.h and paged.h, exported by the same
 * library (libmoe.so): the residual's addition with the RMS norm, products with
 * 4-bit weights, and the choice of the next token.
 *
 * Conventions are those of moe.h: device pointers, caller-owned buffers, calls
 * that only enqueue work on the given stream, argument errors reported before
 * anything is enqueued, the message of a failed call in moe_last_error().
 * Nothing is allocated, no call synchronises and none keeps anything from one
 * call for the next, so calls on several streams at once are independent.
 */
#ifndef SPARSE_MOE_BIT_GB300_STEP_H
#define SPARSE_MOE_BIT_GB300_STEP_H

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { STEP_BF16 = 1, STEP_F16 = 2, STEP_F32 = 3, STEP_E4M3 = 4, STEP_I8 = 5 };

/*
 * The residual's addition and the RMS norm over the features of every row
 * (token t, head h; H = 1 for the stream itself, the number of heads for norms
 * of queries and keys):
 *   s = x + residual (x where residual is NULL)
 *   n = s / sqrt(mean(s^2) + eps) * (weight + (unit_offset ? 1 : 0))
 * all in fp32; `sum` takes s rounded to x's type, y takes n.  n is computed from
 * s before that rounding.  With an 8-bit y, the features of a row in groups of
 * `group` share a scale:
 *   scale = max|n| / 448 (e4m3) or / 127 (int8) in fp32 (below 2^-126 rounded up, so
 *           that y stays in its range; 0 where the group is all zeros, and only there)
 *   y       = fp32's quotient n / scale rounded to nearest, ties to even (0 where scale is)
 * so that y * scale stands for n.  NaN and infinities reach the group's scale
 * (the scale of a group with either is not finite).  Squares are fp32's: of
 * magnitudes above 1e19 the mean is infinite and n is 0, of rows below 1e-22 it is 0
 * and n goes by eps alone (with eps 0 an infinity, and NaN where s is 0).
 * A row's squares are added in an order that goes by d, alignment and whether T * H is below
 * four rows an SM: between a small and a large batch a row's n may differ in fp32's last bits.
 *   x, residual, sum  `dtype` (BF16, F16 or F32) [T][H][d]; features contiguous,
 *           token and head strides in elements.  sum: NULL exactly where
 *           residual is.  sum may be residual or x, and y may be x, with the same
 *           type and strides (in place); otherwise no output may overlap another
 *           array, nor a row of it another row.
 *   weight  dtype or fp32 [d], or NULL (ones; without unit_offset)
 *   y       y_dtype, any of the five
 *   scales  fp32 [T][H][d / group] dense for an 8-bit y, else NULL
 *   group   divides d for an 8-bit y (0: d), else 0
 *   d       1 .. 32768
 */
moe_status rms_norm(const void* x, int dtype, int T, int H, int d, int64_t x_token_stride,
                    int64_t x_head_stride, const void* residual, int64_t r_token_stride,
                    int64_t r_head_stride, void* sum, int64_t s_token_stride,
                    int64_t s_head_stride, const void* weight, int weight_dtype, int unit_offset,
                    float eps, void* y, int y_dtype, int64_t y_token_stride,
                    int64_t y_head_stride, float* scales, int group, void* stream);

/*
 * Products with 4-bit weights, for a decode batch's projections and logits:
 *   y[t][o] = sum_k x[t][k] (scale[o][k / group] * code[o][k] + bias[o][k / group])
 * with codes, scales and biases in moe.h's checkpoint layout (two codes a byte,
 * the even k in the low nibble; nothing is repacked), the products exact and
 * the sums in fp32.
 *   x       [T][K]: BF16 or F16, or E4M3 or I8 with scales: x stands for
 *           x * x_scale[t][k / x_group].  Rows x_token_stride elements apart,
 *           16-byte aligned (the base and every row).
 *           Magnitudes below 2^110; a token that holds a NaN or an infinity has a
 *           y without finite numbers (NaN also where the formula has an infinity)
 *           and changes no other token's.
 *   x_scale fp32 [T][K / x_group] dense for an 8-bit x, else NULL; x_group: K or
 *           a multiple of 64 that divides K (0: K)
 *   codes   uint8 [O][K / 2], scale and bias 16-bit (MOE_SCALE_F16 or _BF16)
 *           [O][K / group], all dense, 16-byte aligned; scales below 2^100
 *   group   a multiple of 64 that divides K
 *   y       BF16, F16 or F32 [T][O], rows y_token_stride elements apart; may not
 *           overlap x, nor one row another
 * Every 16 tokens (8 where K is above 16384) read the weights anew, one after another from
 * L2, and turn them into operands anew.  A matrix product of 16-bit weights, where a caller keeps
 * those too, is the faster one beyond 16 tokens for a projection (2048 -> 5120, weights in L2,
 * 8 tokens 8.6 us here and 6.6 there, 40 13.5 and 6.6, 256 35 and 10), beyond 32 for a vocabulary
 * (2048 -> 131072, 8 tokens 37 and 82, 32 82 and 86, 64 153 and 97, 256 606 and 109): a prompt's
 * products are better served so.  K up to 36864, T up to 524280.  The result does not depend on timing, nor a token's on the others in
 * the call beyond the split that T chooses.
 */
moe_status linear4(const void* x, int x_dtype, int T, int K, int64_t x_token_stride,
                   const float* x_scale, int x_group, const void* codes, const void* scale,
                   const void* bias, int scale_dtype, int O, int group, void* y, int y_dtype,
                   int64_t y_token_stride, void* stream);

/*
 * The next token of every row of logits, from a given random number u in [0, 1).
 * The tokens stand in order of (logit descending, index ascending), with weights
 * w = exp((logit - largest logit) / temperature):
 *   top_k > 0   the first top_k tokens are kept, the others' weights count as 0
 *   top_p < 1   of these the shortest first part whose weights sum to at least
 *               top_p times theirs (one token at least)
 *   min_p > 0   of these the tokens with w >= min_p (of the largest weight, 1)
 * and the token is the first in order of index at which the sum of the kept
 * weights exceeds u times their total.  temperature 0 takes the first token of
 * the order.  Weights are rounded to multiples of 2^-45 and their sums exact:
 * no result depends on timing, on the batch or on how a row is split.
 *   logits   BF16, F16 or F32 [B][V], rows `stride` elements apart.  NaN counts as
 *            -inf; a token at -inf is never taken; +inf share the weight evenly.
 *            A row without any other logit: token -1, logprob NaN.
 *   u, temperature, top_p, min_p  fp32 [B];  top_k int32 [B].  Where one of the
 *            last four is NULL, all_* is every row's (temperature 1, top_k 0, top_p 1
 *            and min_p 0 leave all tokens as they are).  Values out of range are
 *            read as the nearest in it (NaN: as off; temperature NaN, or below 0: 0).
 *   token    int32 [B]
 *   logprob  fp32 [B], or NULL: the logarithm of the probability with which the
 *            token was drawn (0 at temperature 0)
 *   V        1 .. 360448
 */
moe_status sample(const void* logits, int dtype, int B, int V, int64_t stride, const float* u,
                  const float* temperature, const int32_t* top_k, const float* top_p,
                  const float* min_p, float all_temperature, int all_top_k, float all_top_p,
                  float all_min_p, int32_t* token, float* logprob, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_MOE_BIT_GB300_STEP_H */
