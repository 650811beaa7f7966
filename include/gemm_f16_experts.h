/*
 * gemm_f16_experts.h -- which experts a token goes to, the order that brings
 * each expert's rows together for the products of gemm_f16_f8.h, and the
 * weighted sum that puts a token's rows together again.
 *
 * Every function follows the rules of gemm_f16_nt.h (see gemm_f16_f8.h).
 */
#ifndef GEMM_F16_EXPERTS_H
#define GEMM_F16_EXPERTS_H

#include "gemm_f16_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    GEMM_F16_ROUTE_SOFTMAX = 0,      /* a token's scores are its logits' softmax  */
    GEMM_F16_ROUTE_SIGMOID = 1       /* ... their sigmoids                        */
};

/*
 * The choice of T tokens among E experts (1 to 1024), `top` each (1 to 32, at
 * most E).  logits [T, E] fp16 or fp32 (logits_f32), bias fp32 [E] or NULL.
 *
 *   s[e]   softmax or sigmoid of the logits
 *   c[e] = s[e] + bias[e], by which experts are chosen; -inf, never chosen,
 *          where the logit or c[e] is -inf
 *   groups > 1: the experts stand in that many groups of E / groups neighbours
 *          (groups divides E and is at most 64); a group's score is the sum of
 *          its two highest c (one, where only one is not -inf), or with
 *          group_max its highest; only the top_groups highest groups' experts
 *          are considered
 *   experts int32 [T, top]: the highest c, in order; ties, here and among
 *          groups, go to the lowest index; -1 where none is left
 *   weights fp32 [T, top]: scale s[e], divided by the sum of the chosen s +
 *          1e-20 where `renormalize`; 0 for expert -1
 *
 * Scores are computed in 64 bits (two experts' scores are often closer than 32
 * tell apart) and weights rounded once.  A token with a NaN among its logits or
 * its c, or +inf among its logits with softmax, gets experts -1 and weights NaN.
 *
 * The order of the S = T * top slots, slot = token * top + choice:
 *   offsets int32 [E + 1]: expert e's slots stand at positions offsets[e] ..
 *          offsets[e + 1] - 1, in ascending order
 *   rows   int32 [S]: the slot at each position; -1 from offsets[E] on
 *   places int32 [T, top]: the position of each slot; -1 for expert -1
 *
 * gemm_f16_route_workspace: pure host function, the bytes of `workspace` (256-
 * byte aligned) that a call needs, 0 for few tokens.
 *
 * GEMM_F16_INVALID_ARG for sizes outside those above, S above 2^31 - 1024 or a
 * NULL array; GEMM_F16_UNSUPPORTED for arrays not aligned to their elements, or a
 * launch of 2^32 threads (64 a token; 32 up to 128 experts, without groups).
 */
int gemm_f16_route_workspace(int64_t T, int64_t E, int32_t top, int64_t *bytes);
int gemm_f16_route(int64_t T, int64_t E, int32_t top, int32_t scores, int32_t groups,
                   int32_t top_groups, int32_t group_max, int32_t renormalize, double scale,
                   const void *logits, int32_t logits_f32, const void *bias, void *experts,
                   void *weights, void *rows, void *places, void *offsets, void *workspace,
                   int64_t workspace_bytes, hipStream_t stream);

/*
 * The gradient of the logits (of the logits' type) from that of the weights
 * (fp32 [T, top]), for the experts that gemm_f16_route chose: the choice and
 * the bias get none.  Slots with expert -1 count for nothing, whatever dweights
 * holds there; a token with NaN weights gets NaN; a logit of -inf gets 0.
 */
int gemm_f16_route_backward(int64_t T, int64_t E, int32_t top, int32_t scores,
                            int32_t renormalize, double scale, const void *logits,
                            int32_t logits_f32, const void *experts, const void *weights,
                            const void *dweights, void *dlogits, hipStream_t stream);

/*
 * out[t] = sum over choices j of weights[t][j] * y[places[t][j]], fp16 [T, N],
 * for y fp16 [T * top, N]; fp32 sums in the order of j, rounded once.  weights
 * NULL: all 1.  A place outside 0 .. T * top - 1 adds weight * 0.
 *
 * gemm_f16_combine_backward: dy[p] = weights[t][j] * dout[t] at p = places[t][j]
 * (fp32, rounded to fp16), and dweights[t][j] the inner product of dout[t] and y[p], 0
 * for no place; rows of dy that are no slot's place (rows[p] = -1) get +0.
 * weights NULL: all 1.  dweights NULL: not computed, and y is not read.
 *
 * GEMM_F16_UNSUPPORTED for N above 2^31 - 8, misaligned arrays, or a launch of 2^32
 * threads: 64 for each token and 512 columns, backward 64 a slot.
 */
int gemm_f16_combine(int64_t T, int32_t top, int64_t N, const void *y, const void *weights,
                     const void *places, void *out, hipStream_t stream);
int gemm_f16_combine_backward(int64_t T, int32_t top, int64_t N, const void *dout, const void *y,
                              const void *weights, const void *rows, const void *places,
                              void *dy, void *dweights, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_EXPERTS_H */
