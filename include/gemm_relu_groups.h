/*
 * gemm_relu_groups.h -- products of libgemm_relu.so whose rows choose their weights.
 *
 * gemm_relu.h multiplies every row of A by one B.  Here the rows come in groups
 * of consecutive rows, and each group has weights of its own:
 *
 *   gemm_relu_grouped           C[m] = act(A[m] @ B[g(m)])
 *   gemm_relu_grouped_backward  its gradients with respect to A and B
 *   gemm_relu_adapters          C[m] = act(X[m] @ W + s_i (X[m] @ U_i) @ V_i),  i = i(m)
 *
 * act is ReLU (relu = 1; +0.0 for every x that is not > 0, NaN included, as in
 * gemm_relu.h) or the identity (relu = 0).
 *
 * Groups.  `ends` is an int32 array in device memory: group g holds rows
 * ends[g - 1] .. ends[g] - 1 (group 0 starts at row 0), so the running sum of
 * the groups' row counts is the table, and it never visits the host.  A group
 * may be empty.  The entries must not decrease; entries outside [0, M] count
 * as 0 or M.  If they decrease, the outputs are unspecified (nothing outside
 * the outputs is touched).  Rows from ends[groups - 1] on belong to no group.
 *
 * Everything else is as in gemm_relu.h: one 16-bit dtype for all matrices, all
 * dense row-major, fp32 accumulation, round to nearest even; device pointers
 * owned by the caller; work is enqueued on `stream` without waiting, as kernel
 * launches only (no memset, copy or allocation: calls can be captured into a
 * HIP graph); arguments are checked before anything is launched; negative
 * return codes (GEMM_RELU_ERR_*, gemm_relu_strerror).  Matrices need 2-byte
 * alignment, int32 and float arrays 4-byte.  The fastest kernels want row
 * lengths that are multiples of 8 elements and 16-byte aligned matrices, the next
 * ones even lengths and 4-byte alignment.
 *
 * Layouts.  GEMM_RELU_B_KN: weights stored (in, out): B (groups, K, N), W (K, N),
 * U (adapters, K, rank), V (adapters, rank, N).  GEMM_RELU_B_NK: stored (out, in):
 * B (groups, N, K), W (N, K), U (adapters, rank, K), V (adapters, N, rank).
 *
 * Workspace.  Each call takes device memory of at least the bytes that its
 * *_workspace function returns for the same arguments (256-byte aligned, not
 * overlapping any other argument; NULL where that is 0).  Its first
 * GEMM_RELU_GROUPS_COUNTER_BYTES must be zero before the first use; every call
 * that runs to completion leaves them zero, so one buffer serves all calls of
 * one stream, of any shape, and those of gemm_relu_splitk too.  Calls that may
 * overlap in time need different ones.
 * The rest holds partial sums, the adapters' intermediates, the masked gradient
 * and, for large products of odd row lengths, copies of the operands on whole
 * cache lines (as large as the operands); nothing of it is kept between calls.
 *
 * Limits: M, N, K <= 2^20, groups, segments, adapters <= 65535, rank <= 256.
 */
#ifndef GEMM_RELU_GROUPS_H
#define GEMM_RELU_GROUPS_H

#include <stdint.h>

#include "gemm_relu.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_RELU_GROUPS_COUNTER_BYTES ((int64_t)65536)

/* Kernels of the products below (`config_id`).  AUTO picks by size and
 * alignment.  DMA_128 and DMA_64 need rows of an even length and 4-byte aligned
 * operands, DMA_256 multiples of 8 elements and 16-byte alignment; a request that
 * the arguments do not allow falls back to DMA_128 or TILED.  Sums may be added in another order by another kernel. */
enum {
    GEMM_RELU_GROUPS_AUTO = -1,
    GEMM_RELU_GROUPS_TILED = 0,   /* 128x128 tiles staged through registers: any row length and alignment */
    GEMM_RELU_GROUPS_DMA_256 = 1, /* 256x256 tiles, 2 direct-to-LDS stages of 64 k, 8 waves */
    GEMM_RELU_GROUPS_DMA_128 = 2, /* 128x128 tiles, 4 stages, 4 compute waves and 4 that only load */
    GEMM_RELU_GROUPS_DMA_64 = 3,  /* 64x64 tiles, 4 stages, 4 compute waves and 4 that only load */
    GEMM_RELU_GROUPS_STREAM = 4   /* few rows a group: 16 to 64 rows x 32 columns, weights streamed into registers;
                                     any row length and alignment (of the gradients dA's; dB goes as by AUTO) */
};

/*
 * C[m] = act(A[m] @ B[g]) for every row m of group g; rows of no group are set
 * to +0.0.  A (M, K), C (M, N).  M == 0 or N == 0: nothing to do.  K == 0: C is
 * filled with +0.0.
 */
int gemm_relu_grouped(const void* A, const void* B, const int32_t* ends, void* C, int64_t M, int64_t N,
                      int64_t K, int64_t groups, int dtype, int b_layout, int relu, int config_id,
                      void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_relu_grouped_workspace(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype, int b_layout);

/*
 * With D = dC where C > 0 and +0.0 elsewhere (relu = 1), or D = dC (relu = 0;
 * C is not read and may be NULL):
 *
 *   dA[m] = D[m] @ B[g]^T for every row m of group g; +0.0 for rows of no group
 *   dB[g] = sum over the rows m of group g of A[m]^T D[m]; +0.0 for an empty group
 *
 * dA has A's shape and dB has B's (in its layout).  Either may be NULL and is
 * then not computed (dA needs no A, dB no B: those may be NULL too).
 */
int gemm_relu_grouped_backward(const void* dC, const void* C, const void* A, const void* B, const int32_t* ends,
                               void* dA, void* dB, int64_t M, int64_t N, int64_t K, int64_t groups, int dtype,
                               int b_layout, int relu, int config_id, void* workspace, int64_t workspace_bytes,
                               void* stream);
int64_t gemm_relu_grouped_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t groups, int dtype,
                                             int b_layout, int relu);

/*
 * A projection shared by all rows, plus for each segment of rows (one request's
 * tokens) a product of low rank: C[m] = act(X[m] @ W + scales[i] (X[m] @ U_i) @ V_i)
 * where row m is in segment s and i = ids[s].  ids[s] outside [0, adapters)
 * (say -1), and rows of no segment: the projection alone.  `ends` has the
 * segments' ends; `ids` is int32, `scales` float, one per adapter, all in
 * device memory.  X (M, K), C (M, N).
 *
 * The low-rank intermediate X @ U_i is summed and scaled in fp32 and kept as a
 * power of two, one for each row, above the row's largest entry, times a sum of
 * two 16-bit values for each entry.  So it does not overflow, and an entry z is
 * off by at most
 *   bf16: 2^-16 |z|
 *   fp16: 2^-22 |z| + 2^-25 times that power of two (fp16's smallest steps: an
 *         entry 2^-12 of the row's largest keeps 12 bits),
 * which is less than the 24 bits of an fp32 intermediate; the output is rounded
 * to 8 or 11.  The weights of an adapter never reach rows that do not use it,
 * infinities and NaN included; in rows that use it, infinities of V come out as
 * the signs of their products say.
 */
int gemm_relu_adapters(const void* X, const void* W, const void* U, const void* V, const float* scales,
                       const int32_t* ends, const int32_t* ids, void* C, int64_t M, int64_t N, int64_t K,
                       int64_t rank, int64_t adapters, int64_t segments, int dtype, int b_layout, int relu,
                       int config_id, void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_relu_adapters_workspace(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters,
                                     int64_t segments, int dtype, int b_layout);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RELU_GROUPS_H */
