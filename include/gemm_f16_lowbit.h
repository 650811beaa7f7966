/*
 * gemm_f16_lowbit.h -- products of libgemm_f16.so whose second operand is
 * held in 4 or 8 bits, and the kernels that put it in that form.
 *
 * Two forms, for the two places where a linear layer's operand is kept for
 * long and read often:
 *
 *   W4  a weight matrix [N, K], 4-bit codes, one scale for each `group`
 *       consecutive weights of a row (group 32, 64 or 128):
 *           W[j][k] = s[j][k / group] * q[j][k],     q in -8 .. 7
 *   Q8  a matrix of activations [R, N], kept from the forward to the backward
 *       pass, 8-bit codes, one scale for each 32 consecutive values of a row:
 *           X[t][j] = s[t][j / 32] * q[t][j],        q in -127 .. 127
 *
 * Scales are fp16 with few significant bits: 8 for W4, 4 for Q8.  A W4 code
 * has at most 3 significant bits (or is -8) and a Q8 code at most 7, so s * q
 * has at most the 11 of fp16 and is exact in it.  Every kernel below therefore
 * works on the same matrix, whether it multiplies codes and scales the sums,
 * or multiplies scaled codes, or writes the matrix out in fp16 first; results
 * differ only by the order of the fp32 sums.
 *
 * Quantising.  s is the smallest number of that many significant bits, and
 * multiple of 2^-24, whose product with the largest code (7 or 127) reaches
 * the group's largest magnitude (at most 9344 for W4).  A code is x / s
 * rounded to nearest, ties to even; where s * code would pass 65504, the code
 * next to it towards zero (Q8 groups that reach past 65088 only).  A group of
 * zeros has s = 2^-24.  A group that holds an infinity or a NaN gets s = NaN
 * and codes 0: all of it, and every sum that it enters, is NaN.  Columns past
 * K (or N) do not count.
 *
 * Every function follows the rules of gemm_f16_nt.h: device pointers owned by
 * the caller, work enqueued on `stream` for the current device, no allocation,
 * no host synchronisation, no memset (each may be captured into a graph), the
 * same status codes, any host thread.  Results are deterministic.  A status
 * other than GEMM_F16_OK means that nothing was written, except
 * GEMM_F16_LAUNCH_FAILED after a first kernel of a call was enqueued.
 */
#ifndef GEMM_F16_LOWBIT_H
#define GEMM_F16_LOWBIT_H

#include "gemm_f16_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_F16_Q8_GROUP 32

/*
 * W4 storage.  Nb = ceil(N / 16) and Kt = ceil(K / 128); what lies past N or K
 * in a tile has code 0.
 *
 *   words   uint32 [Nb][Kt][64][4]: word j of lane l of tile (b, t) holds the
 *           eight weights of row 16 b + l % 16 at columns
 *           128 t + 32 j + 8 (l / 16) + i, i = 0 .. 7, as q + 8 in the four
 *           bits from 16 (i % 2) + 4 (i / 2).  A tile is 1 KB, in the order in
 *           which a wave's lanes feed the 16 x 16 x 32 MFMA.  16-byte aligned.
 *   scales  fp16 [Nb][128 Kt / group][16]: scale of row 16 b + r and columns
 *           group g ..; 8-byte aligned; finite or NaN, at most 8 significant
 *           bits, and |s * q| at most 65504 (what the two functions below
 *           write; other scales give products rounded in more than one way).
 *           Scales of groups past K and of rows past N do not matter.
 *
 * gemm_f16_w4_sizes: pure host function, the bytes of both arrays.
 * GEMM_F16_INVALID_ARG for NULL outputs, negative sizes or a group other than
 * 32, 64 and 128; GEMM_F16_UNSUPPORTED for N or K above 2^31 - 128 or more than
 * 2^31 - 1 tiles.
 *
 * gemm_f16_w4_quantize: W fp16 [N, K] row-major (any 2-byte alignment) to
 * words and scales.
 *
 * gemm_f16_w4_pack: the same storage from codes int8 [N, K] row-major and
 * in_scales fp16 [N, ceil(K / group)] row-major that another quantiser made.
 * Scales are rounded to 8 significant bits (to nearest, ties to even), which
 * changes each weight of a group by up to 2^-8 of its value.  A group with a
 * code outside -8 .. 7, a scale that is not finite (as given or, from 65408, as
 * rounded), or a product past 65504 gets s = NaN and codes 0.
 *
 * gemm_f16_w4_dequantize: words and scales to W fp16 [N, K] row-major.
 *
 * The arrays of one call must not overlap (GEMM_F16_INVALID_ARG), and each
 * must be aligned as said here, fp16 matrices to 2 bytes
 * (GEMM_F16_UNSUPPORTED).  N = 0 or K = 0: nothing to do, GEMM_F16_OK.
 */
int gemm_f16_w4_sizes(int64_t N, int64_t K, int32_t group,
                      int64_t *words_bytes, int64_t *scales_bytes);
int gemm_f16_w4_quantize(int64_t N, int64_t K, int32_t group, const void *W,
                         void *words, void *scales, hipStream_t stream);
int gemm_f16_w4_pack(int64_t N, int64_t K, int32_t group, const void *codes,
                     const void *in_scales, void *words, void *scales, hipStream_t stream);
int gemm_f16_w4_dequantize(int64_t N, int64_t K, int32_t group, const void *words,
                           const void *scales, void *W, hipStream_t stream);

/*
 * Which kernel a low-bit product runs, and what it needs.
 */
enum {
    /* the operand is written out in fp16 into the workspace and the library's
     * fp16 GEMM (with its own split over K) runs on it */
    GEMM_F16_LOWBIT_DECODE = 0,
    /* the codes go from memory to the matrix units through registers; 4 bits:
     * one pass, no workspace; 8 bits: where the rows of X are split, the
     * ranges' fp32 sums through the workspace */
    GEMM_F16_LOWBIT_STREAM = 1,
    /* tiles of the codes and of A through LDS; where K is split, the ranges'
     * fp32 sums through the workspace */
    GEMM_F16_LOWBIT_TILE = 2
};
typedef struct {
    int32_t kernel;           /* one of the values above                      */
    int32_t block_m;          /* rows of C that a workgroup computes          */
    int32_t block_n;          /* columns of C that a workgroup computes       */
    int32_t waves;            /* 64-lane wavefronts per workgroup             */
    int32_t splits;           /* ranges of K summed apart, 1: no split        */
    int32_t grid;             /* workgroups                                   */
    int64_t workspace_bytes;  /* device memory that the call needs            */
} gemm_f16_lowbit_plan_t;

/*
 * gemm_f16_nt_w4: C = A * W^T, A fp16 [M, K] and C fp16 [M, N] row-major at
 * any 2-byte alignment, W [N, K] in W4 storage; fp32 sums rounded once to fp16.
 *
 * `workspace`: device memory of at least the planned bytes, 256-byte aligned
 * (else GEMM_F16_UNSUPPORTED), overlapping none of the other arrays (else
 * GEMM_F16_INVALID_ARG, as for too few bytes); its contents on entry do not
 * matter.  NULL where the plan needs none.  Concurrent calls need separate
 * workspaces unless they are ordered on one stream.
 *
 * gemm_f16_nt_w4_plan: pure host function.  What gemm_f16_nt_w4 runs on a
 * device with num_cus compute units, for an A that is 16-byte aligned.  Where K
 * is a multiple of 8 and A is not so aligned, sizes planned for the tile kernels
 * are streamed instead, 48 rows of A at a time, without the planned workspace
 * (which is asked for all the same).  The weights are then read again for each
 * 48 rows: some hundreds of rows take several times as long.
 *
 * M = 0 or N = 0: nothing to compute.  K = 0: C is filled with +0.
 * GEMM_F16_UNSUPPORTED for M above 2^31 - 1, for N and K as above, and for
 * sizes that decoding and the fp16 GEMM would run, where that refuses them or
 * a matrix has more than 2^60 values.
 */
int gemm_f16_nt_w4_plan(int64_t M, int64_t N, int64_t K, int32_t group, int32_t num_cus,
                        gemm_f16_lowbit_plan_t *plan);
int gemm_f16_nt_w4(int64_t M, int64_t N, int64_t K, int32_t group, const void *A,
                   const void *words, const void *scales, void *C,
                   void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Q8 storage.  Ng = ceil(N / 32); what lies past N in a row has code 0.
 *
 *   codes   int8 [R][32 Ng] row-major, 16-byte aligned
 *   scales  fp16 [R][Ng] row-major, 2-byte aligned; finite or NaN, at most 4
 *           significant bits, |s * q| at most 65504
 *
 * Each row stands alone: a range of rows is such a matrix too.
 *
 * gemm_f16_q8_quantize: X fp16 [R, N] row-major (any 2-byte alignment) to
 * codes and scales.  gemm_f16_q8_dequantize: the other way.  Overlap,
 * alignment and empty sizes as for W4; GEMM_F16_UNSUPPORTED for R or N above
 * 2^31 - 32 or more than 2^36 codes.
 */
int gemm_f16_q8_quantize(int64_t R, int64_t N, const void *X, void *codes, void *scales,
                         hipStream_t stream);
int gemm_f16_q8_dequantize(int64_t R, int64_t N, const void *codes, const void *scales,
                           void *X, hipStream_t stream);

/*
 * gemm_f16_tn_q8: C = A^T * X, A fp16 [K, M] and C fp16 [M, N] row-major at any
 * 2-byte alignment, X [K, N] in Q8 storage; fp32 sums rounded once to fp16.
 * With A the gradient of a linear layer's output and X its kept input, C is
 * the gradient of its weight (stored [M, N] = [outputs, inputs]).  Workspace,
 * plan and empty sizes as for gemm_f16_nt_w4.
 */
int gemm_f16_tn_q8_plan(int64_t M, int64_t N, int64_t K, int32_t num_cus,
                        gemm_f16_lowbit_plan_t *plan);
int gemm_f16_tn_q8(int64_t M, int64_t N, int64_t K, const void *A, const void *codes,
                   const void *scales, void *C, void *workspace, int64_t workspace_bytes,
                   hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_LOWBIT_H */
