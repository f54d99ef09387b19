/*
 * mi355fused -- the products of a language model with the work around them
 * folded in, for AMD Instinct MI355X (gfx950).
 *
 * Public C ABI of libmi355fused.so, beside mi355gemm.h and with its
 * conventions: row-major matrices with int leading dimensions and 64-bit
 * offsets, device pointers owned by the caller, no allocation, work enqueued
 * on `stream` (a hipStream_t, NULL for the default one) without
 * synchronising, misaligned pointers and leading dimensions never an error,
 * thread-safe calls, GEMM_OK or a GEMM_ERR_* code returned (gemm_status_string
 * of mi355gemm.h names them), nothing enqueued on an error.
 *
 * 16-bit operands are all of the call's `type` (GEMM_TYPE_F16 or
 * GEMM_TYPE_BF16).  Sums, softmax statistics and activations are in fp32; an
 * output is rounded once (nearest, ties to even).  Results repeat bit for bit:
 * there are no atomics.  No output may overlap an input or another output.
 *
 * Sizes M, N and K go up to 2^27; larger ones are GEMM_ERR_BAD_ARG.
 *
 * Workspaces: a call that takes one needs at least the bytes its size query
 * reports for the same arguments (the query looks at the pointers' alignment
 * only), at a 16-byte aligned device address, or NULL when that is 0.  Its
 * kernels write and read it on `stream`, so it must not be in use by other
 * work until they finish: calls that overlap in time, replays of two captured
 * graphs among them, need workspaces of their own.
 */
#ifndef MI355FUSED_H
#define MI355FUSED_H

#include "mi355gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#if defined(MI355FUSED_BUILDING)
#define MI355FUSED_API __attribute__((visibility("default")))
#else
#define MI355FUSED_API
#endif

/*
 * Gated product, the first half of a gated feed-forward block:
 *
 *     G = X * Wg^T,   U = X * Wu^T,   H = act(G) * U   (elementwise)
 *
 *   X       : [M][ldx],  ldx >= max(1, K)    (read)
 *   Wg, Wu  : [N][ldw*], ldw* >= max(1, K)   (read; they may be the two halves
 *             of one matrix)
 *   act     : GEMM_ACT_NONE (act(g) = g), GEMM_ACT_RELU or GEMM_ACT_SILU, on
 *             the unrounded sums
 *   H       : [M][ldh], ldh >= max(1, N)     (written)
 *   G, U    : [M][ldg], [M][ldu], or NULL    (written: the products themselves,
 *             as gemm_gated_bwd takes them)
 *
 * K == 0 gives zero products.  M == 0 or N == 0 is a no-op.
 */
MI355FUSED_API int gemm_gated(int type, int act, int M, int N, int K,
                              const void* X, int ldx,
                              const void* Wg, int ldwg,
                              const void* Wu, int ldwu,
                              void* H, int ldh, void* G, int ldg, void* U, int ldu,
                              void* workspace, unsigned long long workspace_bytes,
                              void* stream);

/* Workspace bytes of gemm_gated: 0 for M <= 64, for few outputs (ceil(M / 64) N
 * up to 10000, or 4000 if a pointer or leading dimension is odd) and for
 * operands of at least 128 rows with K >= 128, K % 8 == 0, 16-byte aligned
 * pointers and leading dimensions that are multiples of 8 (below 2^28);
 * otherwise a padded copy of each operand that is not so.  0 also for arguments
 * the call rejects. */
MI355FUSED_API unsigned long long gemm_gated_workspace(int type, int M, int N, int K,
                                                       const void* X, int ldx,
                                                       const void* Wg, int ldwg,
                                                       const void* Wu, int ldwu);

/*
 * The gradients of gemm_gated.  With dH the gradient of H and G, U the
 * products (16-bit, as gemm_gated stored them):
 *
 *     dG = dH * U * act'(G)      dU = dH * act(G)
 *     dX = dG * Wg + dU * Wu     dWg = dG^T * X     dWu = dU^T * X
 *
 * ReLU's slope at 0 is 0, and NaN where the gate is NaN.  dG and dU are computed in fp32 and rounded to the
 * type for the matrix cores (half a step, 2^-9 relative in bf16 and 2^-12 in
 * fp16, beside the outputs' own rounding); the sums over N and M are fp32.  In
 * fp16 they are rounded times a power of two that brings the largest finite
 * one to 2^14 .. 2^15, by which the sums are divided: none overflows, and only
 * those below 2^-28 of the largest lose bits (2^-39 of it at most).
 *
 *   G, U, dH : [M][ld], ld >= max(1, N)      (read)
 *   dX       : [M][lddx], lddx >= max(1, K), or NULL  (written)
 *   dWg, dWu : [N][ld], ld >= max(1, K), or NULL each (written)
 *
 * X is read only for dWg or dWu, Wg and Wu only for dX; they may be NULL
 * otherwise.  An empty sum (M == 0 for the weights, N == 0 for dX) is zero.
 */
MI355FUSED_API int gemm_gated_bwd(int type, int act, int M, int N, int K,
                                  const void* X, int ldx,
                                  const void* Wg, int ldwg,
                                  const void* Wu, int ldwu,
                                  const void* G, int ldg, const void* U, int ldu,
                                  const void* dH, int lddh,
                                  void* dX, int lddx, void* dWg, int lddwg,
                                  void* dWu, int lddwu,
                                  void* workspace, unsigned long long workspace_bytes,
                                  void* stream);

/* Workspace bytes of gemm_gated_bwd: dG and dU (4 bytes a row and column of H),
 * X transposed, fp32 sums of dX where it has few outputs, and padded copies as
 * for gemm_gated.  want_dx: dX is asked for; want_dw:
 * dWg or dWu is. */
MI355FUSED_API unsigned long long gemm_gated_bwd_workspace(int type, int M, int N, int K,
                                                           const void* X, int ldx,
                                                           const void* Wg, int ldwg,
                                                           const void* Wu, int ldwu,
                                                           int want_dx, int want_dw);

/*
 * Product with 4-bit weights, for the few rows of decode steps:
 *
 *     C = act(X * W^T + bias) + residual
 *     W[n][k] = (q[n][k] - zero[n][k / group]) * scale[n][k / group]
 *
 *   X        : [M][ldx], ldx >= max(1, K)               (read)
 *   Wq       : bytes [N][ldq], ldq >= max(1, ceil(K / 2)): q[n][k] is the low
 *              half of byte k / 2 for even k, the high half for odd k  (read)
 *   group    : K values that share a scale, a multiple of 32; the last group
 *              of a row may be shorter
 *   scales   : 16-bit [N][lds], lds >= max(1, ceil(K / group))  (read)
 *   zeros    : bytes [N][ldz], ldz >= max(1, ceil(K / group)), values 0 .. 15,
 *              or NULL for 8 everywhere                  (read)
 *   bias, act, residual, ldr, C, ldc : as for gemm_ex (residual may be C; ReLU
 *              of NaN is 0)
 *
 * The weights are streamed once for every 64 rows of X, so the time grows in
 * steps of 64 rows: many more rows are faster with gemm_ex on weights that the
 * caller has unpacked to 16 bits.
 * K == 0 gives act(bias) + residual.  M == 0 or N == 0 is a no-op.  A group
 * that is not a positive multiple of 32 is GEMM_ERR_BAD_ARG.
 */
MI355FUSED_API int gemm_w4(int type, int M, int N, int K, int group,
                           const void* X, int ldx,
                           const void* Wq, int ldq,
                           const void* scales, int lds,
                           const void* zeros, int ldz,
                           const void* bias, int act,
                           const void* residual, int ldr,
                           void* C, int ldc, void* stream);

/*
 * Softmax cross entropy of the rows of X * W^T against target columns,
 * without storing the products ("logits") z:
 *
 *     lse[m]  = log(sum_n exp(z[m][n]))
 *     loss[m] = lse[m] - z[m][targets[m]]
 *
 *   X       : [M][ldx], ldx >= max(1, K)          (read)
 *   W       : [N][ldw], ldw >= max(1, K), N >= 1  (read)
 *   targets : 64-bit integers [M]                 (read)
 *   ignore  : rows with this target have loss 0 (their lse is computed)
 *   loss    : float [M]                           (written)
 *   lse     : float [M]                           (written)
 *
 * A target outside [0, N) that is not `ignore` gives a loss of NaN.  M == 0
 * is a no-op; N == 0 with M > 0 is GEMM_ERR_BAD_ARG.
 */
MI355FUSED_API int gemm_xent(int type, int M, int N, int K,
                             const void* X, int ldx, const void* W, int ldw,
                             const long long* targets, long long ignore,
                             float* loss, float* lse,
                             void* workspace, unsigned long long workspace_bytes,
                             void* stream);
MI355FUSED_API unsigned long long gemm_xent_workspace(int type, int M, int N, int K,
                                                      const void* X, int ldx,
                                                      const void* W, int ldw);

/*
 * The gradients of gemm_xent for a gradient dloss of each row's loss:
 *
 *     d[m][n] = (exp(z[m][n] - lse[m]) - [n == targets[m]]) * dloss[m]
 *     dX = d * W     dW = d^T * X
 *
 * computed in pieces of the columns: each piece's d goes to the workspace,
 * rounded to the type after a common factor that brings the largest finite
 * |dloss| to 1 (bf16) or 2^14 (fp16, so that small probabilities do not
 * underflow); the gradients' fp32 sums are divided by it.
 * The sums over N (in fp32 across the pieces) and M are fp32.
 *
 *   lse     : float [M], as gemm_xent stored it   (read)
 *   dloss   : float [M]                           (read)
 *   dX      : [M][lddx], lddx >= max(1, K), or NULL  (written)
 *   dW      : [N][lddw], lddw >= max(1, K), or NULL  (written)
 *
 * Rows with target `ignore` contribute nothing, whatever their X, lse and
 * dloss; a target outside [0, N) that is not `ignore` makes the row's d NaN.
 * M == 0 gives dW = 0; X, W, targets, lse and dloss are then not read and may
 * be NULL.
 */
MI355FUSED_API int gemm_xent_bwd(int type, int M, int N, int K,
                                 const void* X, int ldx, const void* W, int ldw,
                                 const long long* targets, long long ignore,
                                 const float* lse, const float* dloss,
                                 void* dX, int lddx, void* dW, int lddw,
                                 void* workspace, unsigned long long workspace_bytes,
                                 void* stream);
MI355FUSED_API unsigned long long gemm_xent_bwd_workspace(int type, int M, int N, int K,
                                                          const void* X, int ldx,
                                                          const void* W, int ldw,
                                                          int want_dx, int want_dw);

#ifdef __cplusplus
}
#endif

#endif /* MI355FUSED_H */
