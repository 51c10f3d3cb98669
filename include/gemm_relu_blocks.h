/*
 * gemm_relu_blocks.h -- products of libgemm_relu.so on 8-bit floating-point
 * matrices scaled by blocks of 128, and an expert layer for a few tokens.
 *
 *   gemm_relu_quantize_blocks  8-bit values and scales of a 16-bit matrix
 *   gemm_relu_blocks           C = act(A @ B^T) of two such matrices, dense or grouped
 *   gemm_relu_blocks_backward  the gradients of a layer that multiplies so
 *   gemm_relu_experts          a whole expert layer (routing, both products, sum) for up to 64 tokens
 *
 * Quantized matrices.  Values are e4m3 (GEMM_RELU_E4M3: largest 448, one NaN, no
 * infinity) or e5m2 (GEMM_RELU_E5M2: largest 57344, infinities), row-major, with
 * a row pitch in bytes that is a multiple of 16 and at least the row length, from
 * a 16-byte aligned address.  Bytes between a row's end and its pitch are never
 * used.  Scales are dense fp32 arrays in one of two forms:
 *
 *   rows    scales[b][r] (blocks, rows): elements 128 b .. 128 b + 127 of row r
 *   tiles   scales[i][b] (row blocks, blocks): rows 128 i .. of block b
 *
 * An element stands for its value times its scale.  The last block of a row (and
 * the last row block) may be shorter.
 *
 * Everything else is as in gemm_relu.h and gemm_relu_groups.h: 16-bit matrices
 * are fp16 or bf16 and dense, device pointers are owned by the caller, work is
 * enqueued on `stream` without waiting, as kernel launches only (calls can be
 * captured into a HIP graph), arguments are checked before anything is launched,
 * and errors are negative codes.  16-bit matrices need 2-byte alignment, fp32
 * and int32 arrays 4-byte.
 *
 * Workspace.  As in gemm_relu_groups.h (gemm_relu_blocks needs none): device memory of at least the bytes that
 * the *_workspace function returns for the same arguments, 256-byte aligned, its
 * first GEMM_RELU_GROUPS_COUNTER_BYTES zero before the first use and left zero by
 * every call; one buffer serves all calls of one stream, of both headers.
 *
 * Limits: M, N, K <= 2^20, groups, matrices <= 65535, pitches <= 2^21;
 * gemm_relu_experts: tokens <= 64, experts <= 1024, top <= 16, and less than 2^31
 * bytes for the intermediate (4 tokens top hidden) and the partial sums (4 tokens
 * top N, times the parts that K is cut into).
 */
#ifndef GEMM_RELU_BLOCKS_H
#define GEMM_RELU_BLOCKS_H

#include <stdint.h>

#include "gemm_relu.h"
#include "gemm_relu_groups.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_RELU_BLOCK 128

/* Formats of 8-bit matrices. */
enum { GEMM_RELU_E4M3 = 0, GEMM_RELU_E5M2 = 1 };

/* Forms of scales. */
enum { GEMM_RELU_SCALES_ROWS = 0, GEMM_RELU_SCALES_TILES = 1 };

/* Kernels of gemm_relu_blocks (`config_id`): AUTO picks by size. */
enum {
    GEMM_RELU_BLOCKS_AUTO = -1,
    GEMM_RELU_BLOCKS_256 = 0,     /* 256x256 tiles, LDS DMA */
    GEMM_RELU_BLOCKS_128 = 1,     /* 128x128 tiles */
    GEMM_RELU_BLOCKS_64 = 2,      /* 64x64 tiles */
    GEMM_RELU_BLOCKS_STREAM = 3   /* few rows a group, or few operations: 16 to 64 rows x 32 or 64 columns, K cut over waves */
};

/*
 * Quantizes `count` matrices X (count, R, C), each on its own.  With mask (of X's
 * shape, or NULL) an element of X counts as +0.0 where mask is not above zero.
 *
 *   s = max(largest finite magnitude of the block, 2^-80) / largest value of the format
 *   q = s's quotient x / s, rounded to fp32 and then to the format (to nearest even)
 *
 * both divisions correctly rounded; with power_of_two != 0, s is rounded up to a
 * power of two first.  NaN stays NaN; infinities become NaN in e4m3 and stay in
 * e5m2; neither changes its block's scale.
 *
 * Outputs, each pair computed if its Q is not NULL:
 *   Q (count, R, C) at pitch ldq, scales (count, ceil(C/128), R) in form `rows`, or
 *       with form = tiles (count, ceil(R/128), ceil(C/128));
 *   QT (count, C, R) at pitch ldqt, the transposed matrix: scales_t (count, ceil(R/128), C)
 *       in form `rows` (blocks of 128 rows of X), or with form = tiles (count, ceil(C/128),
 *       ceil(R/128)), the same tiles as Q's.
 */
int gemm_relu_quantize_blocks(const void* X, const void* mask, void* Q, float* scales, void* QT, float* scales_t,
                              int64_t count, int64_t R, int64_t C, int64_t ldq, int64_t ldqt, int dtype, int format,
                              int form, int power_of_two, void* stream);

/*
 * C[m] = act(A[m] @ B[g]^T) for every row m of group g (gemm_relu_groups.h: `ends`;
 * NULL with groups = 1: all rows), rows of no group set to +0.0:
 *
 *   C[m][n] = act(sum over blocks b of sa[b][m] sb sum over k in b of A[m][k] B[g][n][k])
 *
 * A (M, K) in format_a at pitch lda with scales in form `rows`; B (groups, N, K) in
 * format_b at pitch ldb with scales in form_b, for each group (rows: (K/128, N);
 * tiles: (N/128, K/128), rounded up); C (M, N) dense, of `dtype`.  The matrix unit
 * adds 8 products of consecutive k at a time, in fixed point: of each it drops what
 * lies below 2^-13 of the largest of the 8.  Those sums, the scaled sums of blocks and
 * all else are fp32, and the product of two scales may lie outside its range where a
 * block's scaled sum does not.  (Sums of products of 16-bit values would keep all bits at half
 * the rate.  Of quantized normal values the dropped bits are 2^-16 of a result, in the
 * 2-norm; its rounding to fp16 is 2^-12, to bf16 2^-9.)
 */
int gemm_relu_blocks(const void* A, const float* scales_a, const void* B, const float* scales_b, const int32_t* ends,
                     void* C, int64_t M, int64_t N, int64_t K, int64_t groups, int64_t lda, int64_t ldb, int format_a,
                     int format_b, int form_b, int dtype, int relu, int config_id, void* stream);

/*
 * Gradients of C = act(X @ W^T), X (M, K), W (N, K), for C's gradient dC, both (M, N)
 * of `dtype`.  With D = dC where C > 0 and +0.0 elsewhere (relu = 1), or D = dC
 * (relu = 0; C is not read and may be NULL), quantized to `format` in blocks of 128
 * along the summed dimension:
 *
 *   dX (M, K) = quantized D @ W     from WT (K, N) in format_w with scales in form tiles
 *   dW (N, K) = quantized D^T @ X   from XT (K, M) in format_x with scales in form rows
 *
 * (gemm_relu_quantize_blocks writes both as its transposed outputs.)  Either output
 * may be NULL and is then not computed, and its operand not read.
 */
int gemm_relu_blocks_backward(const void* dC, const void* C, const void* XT, const float* scales_xt, const void* WT,
                              const float* scales_wt, void* dX, void* dW, int64_t M, int64_t N, int64_t K, int64_t ldxt,
                              int64_t ldwt, int format, int format_x, int format_w, int dtype, int relu, void* workspace,
                              int64_t workspace_bytes, void* stream);
int64_t gemm_relu_blocks_backward_workspace(int64_t M, int64_t N, int64_t K);

/*
 * Y[t] = sum over t's choices j of weights[t][j] (ReLU(X[t] @ W1[e]) @ W2[e]), e = ids[t][j].
 *
 * With logits (tokens, experts) not NULL the choices are made here and written to
 * ids and weights (tokens, top): the `top` largest logits of a token, the largest
 * first, ties to the lowest index; logits of -inf are never chosen (a token that
 * has fewer others gets id -1 with weight 0 for the rest).  Weights are the softmax
 * over the token's logits, or over its chosen ones (renormalize = 1).  A token with
 * a logit of NaN or +inf gets ids -1, weights NaN and a row of NaN.
 * With logits NULL ids and weights are read; ids outside [0, experts) are skipped.
 * A token without a choice gets a row of +0.0.
 *
 * X (tokens, K), Y (tokens, N), fp16 or bf16.  Weights of X's dtype (format = -1):
 * W1 (experts, hidden, K), W2 (experts, N, hidden) with b_layout = GEMM_RELU_B_NK, or
 * (experts, K, hidden) and (experts, hidden, N) with GEMM_RELU_B_KN, dense.  8-bit
 * weights (format = GEMM_RELU_E4M3 or _E5M2): GEMM_RELU_B_NK, at pitches ld1 and ld2,
 * with scales in form tiles; they are multiplied as they are, X is not quantized.
 *
 * weights[t][j] ReLU(..) is computed in fp32 and kept as a sum of two values of X's
 * dtype, off by at most 2^-16 (bf16) or 2^-22 (fp16) of the value, or 2^-134 and 2^-25;
 * fp16 values past 65504 are infinite, as in a layer of two products.
 */
int gemm_relu_experts(const void* X, const void* W1, const float* scales1, const void* W2, const float* scales2,
                      const float* logits, int32_t* ids, float* weights, void* Y, int64_t tokens, int64_t N,
                      int64_t K, int64_t hidden, int64_t experts, int64_t top, int64_t ld1, int64_t ld2, int renormalize,
                      int dtype, int format, int b_layout, void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_relu_experts_workspace(int64_t tokens, int64_t N, int64_t hidden, int64_t experts, int64_t top, int b_layout);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RELU_BLOCKS_H */
