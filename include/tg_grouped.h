/*
 * tg_grouped.h — products of rows grouped by expert with their expert's weight,
 * and their gradients (libtg_gemm.so, MI355X / gfx950).
 *
 * X (M×K) holds rows sorted by expert, W one weight (N×K, stored as tg_gemm's B)
 * for each of E experts.  `ends` says where each expert's rows end: expert e has
 * the rows ends[e−1] <= i < ends[e], with ends[−1] = 0.
 *
 *     Y[i]  = X[i]·W[e]ᵀ          rows of expert e
 *     dX[i] = dY[i]·W[e]
 *     dW[e] = Σ_i dY[i]ᵀ·X[i]     over the rows of expert e, 0 where it has none
 *
 * Rows from ends[E−1] on belong to no expert: what they hold reaches nothing, and their
 * rows of Y and dX are 0.  `ends` lies in device memory and is read there, so that a
 * router's counts never pass through the host.  Whatever it holds, nothing outside
 * the arrays is touched: a value counts as at least the one before it, and
 * as 0 to M.
 *
 * Operands and results are binary16 or bfloat16; products are exact, summed in
 * fp32 and rounded once to nearest even.  Results do not depend on the order in
 * which workgroups run: repeated calls give the same bits.  What a row holds (NaN
 * and infinity included) reaches its own row of Y and dX and its expert's dW alone.
 */
#ifndef TG_GROUPED_H
#define TG_GROUPED_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The product a plan or a workspace is asked for. */
enum { TG_GROUPED_Y = 0, TG_GROUPED_DX = 1, TG_GROUPED_DW = 2 };

/*
 * tg_grouped_workspace_bytes — device memory that a call needs as workspace
 * (host-only); -1 if the arguments would be refused.  `product` is one of the above; A and
 * B with their leading dimensions are the call's first two operands: X and W (Y),
 * dY and W (DX), dY and X (DW).  Operands that have no 16-byte aligned rows, or N or K
 * that is no multiple of 8, are copied into it first, and sums over K, N or the rows
 * that are cut into parts leave these there in fp32; 0 where neither is so.
 * A workspace holds nothing between calls; calls that may overlap must not share one.
 */
int64_t tg_grouped_workspace_bytes(int product, const void *A, const void *B, int64_t M, int64_t E, int64_t N,
                                   int64_t K, int64_t lda, int64_t ldb, int64_t w_stride);

/*
 * tg_grouped_f16, tg_grouped_bf16 — enqueue Y.
 *
 *   X, W, Y   device pointers; row i of X at X + i·ldx, row n of expert e's weight
 *             at W + e·w_stride + n·ldw, row i of Y at Y + i·ldy (elements).  ldx,
 *             ldw >= K, ldy >= N; w_stride >= 0 (not looked at for E <= 1).  Any
 *             alignment of an element is accepted.  Y must not overlap what is
 *             read (not checked).
 *   ends      device pointer to E 64-bit integers.
 *   workspace device memory, 256-byte aligned, of at least
 *             tg_grouped_workspace_bytes(TG_GROUPED_Y, X, W, ...) bytes; NULL where
 *             that is 0.
 *   stream    hipStream_t.  Only kernels are launched: the call may be recorded
 *             into a graph, whose replays read `ends` anew.
 *
 * M == 0 or N == 0: nothing happens.  E == 0 or K == 0: Y is set to 0.  Returns TG_OK,
 * TG_ERR_INVALID_ARG (negative sizes, a leading dimension too small, a NULL or
 * misaligned pointer with elements behind it, a workspace that is NULL, misaligned
 * or too small), TG_ERR_TOO_LARGE (M >= 2^31, E >= 2^16, N or K >= 2^21, a leading
 * dimension >= 2^31, w_stride >= 2^42 or a product of 2^23 or more tiles, which
 * are of 16×32 to 256×256), TG_ERR_DEVICE or TG_ERR_LAUNCH.
 */
int tg_grouped_f16(const void *X, const void *W, const int64_t *ends, void *Y, int64_t M, int64_t E, int64_t N,
                   int64_t K, int64_t ldx, int64_t ldw, int64_t w_stride, int64_t ldy, void *workspace,
                   int64_t workspace_bytes, void *stream);
int tg_grouped_bf16(const void *X, const void *W, const int64_t *ends, void *Y, int64_t M, int64_t E, int64_t N,
                    int64_t K, int64_t ldx, int64_t ldw, int64_t w_stride, int64_t ldy, void *workspace,
                    int64_t workspace_bytes, void *stream);

/*
 * tg_grouped_dx_f16, tg_grouped_dx_bf16 — enqueue dX (M×K, row i at dX + i·lddx),
 * with a workspace for (TG_GROUPED_DX, dY, W, ...).  M == 0 or K == 0: nothing
 * happens.  E == 0 or N == 0: dX is set to 0.  Status codes as above.
 */
int tg_grouped_dx_f16(const void *dY, const void *W, const int64_t *ends, void *dX, int64_t M, int64_t E, int64_t N,
                      int64_t K, int64_t lddy, int64_t ldw, int64_t w_stride, int64_t lddx, void *workspace,
                      int64_t workspace_bytes, void *stream);
int tg_grouped_dx_bf16(const void *dY, const void *W, const int64_t *ends, void *dX, int64_t M, int64_t E,
                       int64_t N, int64_t K, int64_t lddy, int64_t ldw, int64_t w_stride, int64_t lddx,
                       void *workspace, int64_t workspace_bytes, void *stream);

/*
 * tg_grouped_dw_f16, tg_grouped_dw_bf16 — enqueue dW (row n of expert e at
 * dW + e·dw_stride + n·lddw, dw_stride >= (N − 1)·lddw + K for E > 1), with a
 * workspace for (TG_GROUPED_DW, dY, X, ..., w_stride not looked at).  E, N or K == 0: nothing
 * happens.  M == 0: dW is set to 0.  Status codes as above, TG_ERR_TOO_LARGE also for
 * M >= 2^31 − 256.
 */
int tg_grouped_dw_f16(const void *dY, const void *X, const int64_t *ends, void *dW, int64_t M, int64_t E, int64_t N,
                      int64_t K, int64_t lddy, int64_t ldx, int64_t lddw, int64_t dw_stride, void *workspace,
                      int64_t workspace_bytes, void *stream);
int tg_grouped_dw_bf16(const void *dY, const void *X, const int64_t *ends, void *dW, int64_t M, int64_t E, int64_t N,
                       int64_t K, int64_t lddy, int64_t ldx, int64_t lddw, int64_t dw_stride, void *workspace,
                       int64_t workspace_bytes, void *stream);

/*
 * tg_grouped_plan — host-only: the kernels that a call for `product` would use
 * (names separated by spaces, truncated to name_len bytes with the NUL; empty where
 * nothing would be launched); arguments as for tg_grouped_workspace_bytes.  Returns the
 * argument-validation status.
 */
int tg_grouped_plan(int product, const void *A, const void *B, int64_t M, int64_t E, int64_t N, int64_t K,
                    int64_t lda, int64_t ldb, int64_t w_stride, char *name, int64_t name_len);

#ifdef __cplusplus
}
#endif

#endif /* TG_GROUPED_H */
