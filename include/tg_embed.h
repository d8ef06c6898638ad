/*
 * tg_embed.h — embedding lookup with scaling, and its gradient
 * (libtg_gemm.so, MI355X / gfx950).
 *
 *     Y[i] = scale·W[tokens[i]]                    W: V×K, Y: M×K
 *     dW[v] = scale·Σ_{i: tokens[i] = v} dY[i]
 *
 * A product with scale is taken in fp32 and rounded once; dW is summed in fp32, in
 * the order of the rows of dY, and rounded once.  Results do not depend on the
 * order in which workgroups run: repeated calls give the same bits.
 *
 * A token outside [0, V) makes its row of Y NaN and adds nothing to dW.  A row of
 * dW that no token names is 0, and so is row `padding`, whatever names it.
 */
#ifndef TG_EMBED_H
#define TG_EMBED_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * tg_embedding_f32, _f16, _bf16 — enqueue the lookup.
 *
 *   tokens   device pointer to M 64-bit integers.
 *   W        device pointer, row v at W + v·ldw (elements), ldw >= K (any for
 *            V <= 1).
 *   Y        device pointer, row i at Y + i·ldy, of W's type; overwritten.  It must
 *            not overlap W or tokens (not checked).
 *   stream   hipStream_t.  One kernel is launched: the call may be recorded into
 *            a graph.
 *
 * Any alignment of an element is accepted.  M == 0 or K == 0: nothing happens.
 * V may be 0 (every token is outside then).  Returns TG_OK, TG_ERR_INVALID_ARG
 * (negative sizes, a leading dimension below K, a NULL pointer with elements
 * behind it), TG_ERR_TOO_LARGE (M, V, K, ldw or ldy >= 2^31, or M·K >= 2^40),
 * TG_ERR_DEVICE or TG_ERR_LAUNCH.
 */
int tg_embedding_f32(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K, int64_t ldw,
                     int64_t ldy, float scale, void *stream);
int tg_embedding_f16(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K, int64_t ldw,
                     int64_t ldy, float scale, void *stream);
int tg_embedding_bf16(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K, int64_t ldw,
                      int64_t ldy, float scale, void *stream);

/* tg_embedding_bwd_workspace_bytes — device memory a backward call needs as
 * workspace (host-only); -1 if the sizes would be refused.  It holds nothing
 * between calls; calls that may overlap must not share one. */
int64_t tg_embedding_bwd_workspace_bytes(int64_t M, int64_t V, int64_t K);

/*
 * tg_embedding_bwd_f32, _f16, _bf16 — enqueue dW.
 *
 *   dY       device pointer, row i at dY + i·lddy, lddy >= K (any for M <= 1).
 *   dW       device pointer, row v at dW + v·lddw, of dY's type; rows [0, V) and
 *            columns [0, K) are overwritten, nothing else is touched.
 *   padding  the row that gets no gradient; any value outside [0, V): none.
 *   workspace  device memory, 256-byte aligned, of at least
 *            tg_embedding_bwd_workspace_bytes(M, V, K) bytes.
 *
 * Only kernels are launched.  V == 0 or K == 0: nothing happens; M == 0: dW is set
 * to 0.  Status codes as above, TG_ERR_INVALID_ARG also for a workspace that is
 * NULL, misaligned or too small, TG_ERR_TOO_LARGE also for M + V >= 2^31 − 64
 * or (M + V)·K >= 2^40.
 */
int tg_embedding_bwd_f32(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K,
                         int64_t lddy, int64_t lddw, float scale, int64_t padding, void *workspace,
                         int64_t workspace_bytes, void *stream);
int tg_embedding_bwd_f16(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K,
                         int64_t lddy, int64_t lddw, float scale, int64_t padding, void *workspace,
                         int64_t workspace_bytes, void *stream);
int tg_embedding_bwd_bf16(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K,
                          int64_t lddy, int64_t lddw, float scale, int64_t padding, void *workspace,
                          int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TG_EMBED_H */
