/*
 * mi355tune -- what fine tuning needs next to a model's products: low-rank
 * adapters beside a shared projection, their gradients, and updates
 * orthogonalised by Newton-Schulz products, for AMD Instinct MI355X (gfx950).
 *
 * Public C ABI of libmi355tune.so, beside mi355gemm.h and mi355fused.h and with
 * their conventions: row-major matrices with int leading dimensions and 64-bit
 * offsets, device pointers owned by the caller, no allocation, work enqueued
 * on `stream` (a hipStream_t, NULL for the default one) without
 * synchronising, misaligned pointers and leading dimensions never an error,
 * thread-safe calls, GEMM_OK or a GEMM_ERR_* code returned (gemm_status_string
 * of mi355gemm.h names them), nothing enqueued on an error.
 *
 * Sums are in fp32 or more; an output is rounded once (nearest, ties to even).
 * Results repeat bit for bit: nothing is summed in an order that changes.  No
 * output may overlap an input or another output, except where a call says so.
 *
 * Workspaces: a call that takes one needs at least the bytes its size query
 * reports for the same arguments, at a 16-byte aligned device address, or NULL
 * when that is 0.  Its kernels write and read it on `stream`, so it must not be
 * in use by other work until they finish: calls that overlap in time, replays
 * of two captured graphs among them, need workspaces of their own.  What it
 * held before does not matter.
 */
#ifndef MI355TUNE_H
#define MI355TUNE_H

#include "mi355gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#if defined(MI355TUNE_BUILDING)
#define MI355TUNE_API __attribute__((visibility("default")))
#else
#define MI355TUNE_API
#endif

/*
 * A projection shared by all rows beside the low-rank adapter that each row
 * names:
 *
 *     t[m] = X[m] * A[a]^T,  a = ids[m]
 *     C[m] = act(X[m] * W^T + scales[a] * t[m] * B[a]^T + bias) + residual[m]
 *
 *   type    : GEMM_TYPE_F16 or GEMM_TYPE_BF16, of X, W, A, B, bias, residual, C
 *   X       : [M][ldx], ldx >= max(1, K)                            (read)
 *   W       : [N][ldw], ldw >= max(1, K)                            (read)
 *   A       : [S][R][lda], lda >= max(1, K), adapters stride_a elements
 *             apart                                                 (read)
 *   B       : [S][N][ldb], ldb >= R, adapters stride_b apart        (read)
 *   ids     : 64-bit integers [M], in any order: the row's adapter, below 0 for
 *             none (the projection alone); S and more make the row of C NaN
 *   scales  : float [S], or NULL for 1 everywhere                   (read)
 *   bias, act, residual, ldr, C, ldc : as for gemm_ex (residual may be C; ReLU
 *             of NaN is NaN)
 *   T       : float [M][ldt], ldt >= R, or NULL: t, as gemm_lora_bwd takes it;
 *             0 for rows without an adapter, NaN for unknown ones   (written)
 *
 * t is an operand of the second product in two 16-bit values of the type, within
 * 2^-15 (bf16) or 2^-21 (fp16, and 2^-37 of the largest of its 16 ranks) of itself,
 * so C is rounded once.  An adapter of fewer ranks than R has zeros in the others.
 * What one row's adapter holds, infinities and NaN too, reaches no other row.
 *
 * Rows whose neighbours have the same adapter share its reads; in any other
 * order each block of 16 rows reads every adapter that it names.
 *
 * R is 1 .. 1024, M, N, K and S go up to 2^27; others are GEMM_ERR_BAD_ARG.
 * K == 0 gives act(bias) + residual.  M == 0 is a no-op, and so is N == 0
 * without T.
 */
MI355TUNE_API int gemm_lora(int type, int M, int N, int K, int R, int S,
                            const void* X, int ldx, const void* W, int ldw,
                            const void* A, int lda, long long stride_a,
                            const void* B, int ldb, long long stride_b,
                            const long long* ids, const float* scales,
                            const void* bias, int act, const void* residual, int ldr,
                            void* C, int ldc, float* T, int ldt,
                            void* workspace, unsigned long long workspace_bytes,
                            void* stream);

/* Workspace bytes of gemm_lora: t (4 bytes a row and rank, ranks in blocks of
 * 16), and, for many rows, padded copies of X and W where they are not whole
 * 16-byte rows (as for gemm_gated) and of B where R % 8 != 0 or ldb >= 2^22. */
MI355TUNE_API unsigned long long gemm_lora_workspace(int type, int M, int N, int K, int R, int S,
                                                     const void* X, int ldx,
                                                     const void* W, int ldw, int ldb);

/*
 * The gradients of gemm_lora without an activation, for the gradient dC of its
 * result and the T it stored; W is frozen:
 *
 *     dt[m] = scales[a] * dC[m] * B[a]          a = ids[m]
 *     dX[m] = dC[m] * W + dt[m] * A[a]
 *     dA[a] = sum over the rows of a: dt[m]^T * X[m]
 *     dB[a] = scales[a] * sum over the rows of a: dC[m]^T * T[m]
 *
 *   dC      : [M][lddc], lddc >= max(1, N)                          (read)
 *   dX      : [M][lddx], lddx >= max(1, K), or NULL                 (written)
 *   dA, dB  : laid out like A and B, or NULL each; adapters must not
 *             overlap                                               (written)
 *
 * dt and T are operands in two 16-bit values, as t above; in dA and dB the largest
 * is that of all ranks of 32 of an adapter's rows.  Sums over rows, K and N are
 * fp32.  Rows without an adapter (any id below 0, or S and more) reach no adapter's
 * gradient, whatever they hold; an id of S and more makes the row of dX NaN.  An
 * adapter without rows has gradients of zero.
 *
 * For dA and dB, M * min(M, S) goes up to 2^40 (rows are looked for adapter by
 * adapter); more is GEMM_ERR_BAD_ARG.
 *
 * X is read only for dA, T only for dB, W and A only for dX, B for dX and dA;
 * they may be NULL otherwise.  An empty sum is zero.
 */
MI355TUNE_API int gemm_lora_bwd(int type, int M, int N, int K, int R, int S,
                                const void* X, int ldx, const void* W, int ldw,
                                const void* A, int lda, long long stride_a,
                                const void* B, int ldb, long long stride_b,
                                const long long* ids, const float* scales,
                                const float* T, int ldt, const void* dC, int lddc,
                                void* dX, int lddx,
                                void* dA, int ldda, long long stride_da,
                                void* dB, int lddb, long long stride_db,
                                void* workspace, unsigned long long workspace_bytes,
                                void* stream);

/* Workspace bytes of gemm_lora_bwd: B and A with rows and columns exchanged, dt,
 * the rows listed by adapter, dt and T in their order, fp32 sums of adapters'
 * parts and (few rows) of dX over ranges of N, and padded copies of dC and W.
 * want_*: the gradient is asked for. */
MI355TUNE_API unsigned long long gemm_lora_bwd_workspace(int type, int M, int N, int K, int R,
                                                         int S, const void* dC, int lddc,
                                                         const void* W, int ldw, int want_dx,
                                                         int want_da, int want_db);

/* Beside GEMM_TYPE_F16 and GEMM_TYPE_BF16, for gemm_ortho only. */
enum { GEMM_TYPE_F32 = 2 };

/*
 * An update orthogonalised by Newton-Schulz products, as the Muon optimiser
 * does, for L matrices of m x n:
 *
 *     X = G / (|G| + eps)                       (|G|: Frobenius norm)
 *     X = a_k X + b_k (X X^T) X + c_k (X X^T)^2 X     for k = 0 .. steps - 1
 *     O = X
 *
 *   G       : [L][m][ldg], type_g (F32, F16 or BF16), ldg >= max(1, n), matrices
 *             stride_g elements apart                              (read)
 *   coeffs  : 3 * steps floats a_0, b_0, c_0, a_1, ... in HOST memory, read
 *             during the call
 *   O       : [L][m][ldo], type_o (F32, F16 or BF16), matrices stride_o elements
 *             apart, which must not overlap                        (written)
 *
 * m and n may be in either order: the products are taken over the longer side.
 * A G of zeros gives zeros, one with an infinity or NaN gives NaN throughout;
 * neither touches the other matrices.
 *
 * Products are on the 16-bit matrix cores, of values held in two binary16 ones (22
 * bits) at three products for one; for BF16 outputs of large matrices one value
 * is enough for all but the first three iterates.  In the 2-norm the result differs
 * from the formula's by about 2^-19 where G's singular values are of one size, as
 * of noise, by 2^-17 where they spread over a factor of 300 and by 2^-14 where a few
 * are a thousand times the rest, or there (values in one) by 0.12 %, beside the
 * output's own rounding (of 0.17 % in bf16): an F32 result is the most that can be
 * asked for.  This holds for any eps, far above |G| too.  The singular values of
 * every X must stay below 7, as they do for coefficients that converge from [0, 1].
 *
 * steps is 1 .. 64; m, n and L go up to 2^16; others are GEMM_ERR_BAD_ARG, as is
 * a negative or NaN eps.  L == 0, m == 0 or n == 0 is a no-op.
 */
MI355TUNE_API int gemm_ortho(int type_g, int type_o, int L, int m, int n,
                             const void* G, int ldg, long long stride_g,
                             int steps, const float* coeffs, float eps,
                             void* O, int ldo, long long stride_o,
                             void* workspace, unsigned long long workspace_bytes,
                             void* stream);

/* Workspace bytes of gemm_ortho: with s = min(m, n), t = max(m, n), padded to
 * multiples of 64 (128 at least for the large ones), 4 to 16 bytes for each of
 * L * s * t, 4 to 8 for each of L * s * s, fp32 sums of products over a long
 * side, and the norms. */
MI355TUNE_API unsigned long long gemm_ortho_workspace(int type_g, int type_o, int L, int m, int n,
                                                      int steps);

#ifdef __cplusplus
}
#endif

#endif /* MI355TUNE_H */
