/*
 * tg_xent.h — softmax cross entropy of a vocabulary projection, with its
 * gradients, without keeping the logits (libtg_gemm.so, MI355X / gfx950).
 *
 * H (M×K, one row per token) and W (V×K, one row per vocabulary entry) are
 * the operands tg_gemm_f16 / tg_gemm_bf16 multiply: z = H·Wᵀ are the logits.
 * For a token i with target t_i:
 *
 *     lse_i  = log Σ_j exp(z_ij)
 *     loss_i = lse_i − z_i,t_i            (0 for an ignored token)
 *
 * and, for upstream gradients g_i of loss_i and l_i of lse_i,
 *
 *     G_ij = (g_i + l_i)·exp(z_ij − lse_i) − g_i·[j = t_i]
 *     dH   = G·W,      dW = Gᵀ·H.
 *
 * The logits are products of the 16-bit operands summed in fp32; maxima,
 * sums, lse and losses are fp32.  For the gradients the logits are computed
 * again, a piece of the vocabulary at a time; G, scaled so that the largest of
 * its coefficients (g_i and g_i + l_i) is 1 (2^14 for binary16, whose exponent range
 * would flush small probabilities), is rounded once to the operands' type, as the
 * matrix cores take it; dH and dW are summed in fp32 and rounded once.  Against
 * gradients of an unrounded G that is 1.9e-3 for bfloat16 instead of 1.66e-3, the
 * result's own rounding, and 2.5e-4 instead of 2.1e-4 for binary16; where few
 * tokens or words make up an element the two roundings come to 2.4e-3 and 3e-4.
 * One scale serves all tokens: in binary16 an element of G below 2^-28 of the
 * largest coefficient errs by up to 2^-39 of it, so the row of dH of a token whose
 * weight is far below another's is inexact (50001 words: 4e-4 off at 1e-6 of the
 * largest weight, 5e-3 at 1e-7, 4e-2 at 1e-8).
 *
 * Results do not depend on the order in which workgroups run: repeated calls
 * give the same bits.
 */
#ifndef TG_XENT_H
#define TG_XENT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* What `loss` holds, and what the upstream gradient `dloss` refers to.  An
 * ignored token is not counted; with no counted token sum and mean are 0. */
enum {
    TG_XENT_NONE = 0, /* M values, one per token */
    TG_XENT_SUM = 1,  /* one value: the sum */
    TG_XENT_MEAN = 2  /* one value: the sum divided by the number of tokens not ignored */
};

/*
 * tg_xent_workspace_bytes, tg_xent_bwd_workspace_bytes — device memory a call
 * needs as workspace (host-only; the same arguments as the call's).  A
 * workspace holds nothing between calls; calls that may overlap must not
 * share one.  -1 if the arguments would be refused.
 */
int64_t tg_xent_workspace_bytes(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh,
                                int64_t ldw);
int64_t tg_xent_bwd_workspace_bytes(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh,
                                    int64_t ldw);

/*
 * tg_xent_f16, tg_xent_bf16 — enqueue loss and lse.
 *
 *   H, W      device pointers to binary16 / bfloat16, row i of H at H + i·ldh,
 *             row j of W at W + j·ldw (elements).  Any alignment and any
 *             ldh, ldw >= K is accepted; rows that are not 16-byte aligned (or
 *             K not a multiple of 8) are first copied into the workspace.
 *   target    device pointer to M 64-bit targets.  `ignore_index` marks a
 *             token that takes no part: its loss and lse are 0, its row of H
 *             is never read into a result.  Any other target outside [0, V)
 *             makes that token's loss NaN (and its gradients NaN).
 *   loss      device pointer to M floats (TG_XENT_NONE) or one (SUM, MEAN).
 *   lse       device pointer to M floats, or NULL.
 *   workspace device memory, 256-byte aligned, of at least
 *             tg_xent_workspace_bytes(...) bytes.
 *   stream    hipStream_t.  Only kernels are launched: the call may be
 *             recorded into a graph.
 *
 * M == 0: loss (SUM, MEAN) is set to 0.  V and K must be at least 1 where M is
 * not 0.  Returns TG_OK, TG_ERR_INVALID_ARG (negative sizes, a leading
 * dimension below K, V or K 0, a NULL pointer, an unknown reduction, a
 * workspace that is NULL, misaligned or too small), TG_ERR_TOO_LARGE
 * (M >= 2^25, V >= 2^30, K > 2^21, ldh or ldw >= 2^31, or a product of
 * 2^23 or more tiles, which are of 64×64 to 256×256), TG_ERR_DEVICE or
 * TG_ERR_LAUNCH.
 */
int tg_xent_f16(const void *H, const void *W, const int64_t *target, float *loss, float *lse, int64_t M, int64_t V,
                int64_t K, int64_t ldh, int64_t ldw, int64_t ignore_index, int reduction, void *workspace,
                int64_t workspace_bytes, void *stream);
int tg_xent_bf16(const void *H, const void *W, const int64_t *target, float *loss, float *lse, int64_t M, int64_t V,
                 int64_t K, int64_t ldh, int64_t ldw, int64_t ignore_index, int reduction, void *workspace,
                 int64_t workspace_bytes, void *stream);

/*
 * tg_xent_bwd_f16, tg_xent_bwd_bf16 — enqueue dH and dW.
 *
 *   H, W, target, ignore_index, reduction   as for the forward call.
 *   lse       the forward call's lse (M floats).
 *   dloss     device pointer to the upstream gradient of `loss`: M floats
 *             (TG_XENT_NONE) or one (SUM, MEAN).
 *   dlse      upstream gradient of lse, M floats, or NULL for none.
 *   dH        M×K, row i at dH + i·lddh, or NULL if not wanted; an ignored
 *             token's row is set to 0.
 *   dW        V×K, row j at dW + j·lddw, or NULL.
 *             dH and dW have the operands' type and are overwritten.
 *   workspace of at least tg_xent_bwd_workspace_bytes(...) bytes.
 *
 * M == 0: dW is set to 0.  Status codes as for the forward call.
 */
int tg_xent_bwd_f16(const void *H, const void *W, const int64_t *target, const float *lse, const float *dloss,
                    const float *dlse, void *dH, void *dW, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
                    int64_t lddh, int64_t lddw, int64_t ignore_index, int reduction, void *workspace,
                    int64_t workspace_bytes, void *stream);
int tg_xent_bwd_bf16(const void *H, const void *W, const int64_t *target, const float *lse, const float *dloss,
                     const float *dlse, void *dH, void *dW, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
                     int64_t lddh, int64_t lddw, int64_t ignore_index, int reduction, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * tg_xent_plan — host-only: the kernels a forward (backward == 0) or backward
 * call would use for these sizes (names separated by spaces, truncated to
 * name_len bytes with the NUL) and the number of vocabulary pieces.  Returns
 * the argument-validation status.
 */
int tg_xent_plan(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
                 int backward, char *name, int64_t name_len, int64_t *pieces);

#ifdef __cplusplus
}
#endif

#endif /* TG_XENT_H */
