/*
 * tg_ortho.h — orthogonalised update of a projection's weight by a
 * Newton–Schulz iteration (libtg_gemm.so, MI355X / gfx950).
 *
 * For each of `batch` matrices G (rows × cols):
 *
 *     X ← G / (‖G‖_F + eps)
 *     steps times:  A = X·Xᵀ,  B = b·A + c·A²,  X ← a·X + B·X
 *
 * with (a, b, c) per step; for rows > cols the products are taken on the
 * other side (A = Xᵀ·X, X ← a·X + X·B), which is the same X.  The singular
 * vectors stay, each singular value s becomes p(…p(s)) with p(s) = a·s + b·s³ +
 * c·s⁵; the default coefficients (3.4445, −4.7750, 2.0315) bring those above
 * about 1e-3 of ‖G‖_F to [0.7, 1.2] in five steps.
 *
 * Precision.  X is carried in fp32.  The products run on the matrix cores
 * with fp32 sums and binary16 operands under fixed power-of-two scales (X
 * times 2^14, A and B times 2^12), so that every operand keeps 11 significant
 * bits at any magnitude met; the diagonals of A and B, which hold most of
 * their weight, stay in fp32 outside the products.  The result is bfloat16,
 * rounded once, which by itself is 1.66e-3 of the 64-bit result (2-norm, root
 * mean square; at most 2^-8).
 *
 * A direction with a small part of the norm is amplified by up to 485 in five
 * steps, and with it the part of the operands' rounding that falls there.  Up to 64
 * rows of the shorter side every operand is therefore the sum of two binary16
 * values (22 bits), and the result within 2^-8 of the 64-bit one at any spectrum.
 * Above 64 one value is held, and the error depends on the spectrum:
 *
 *     noise, 1/k, singular values from 1 to 1e-2          up to 1.9e-3
 *     noise of 5e-2; of 1e-2 beside eight directions      up to 1.9e-3; 2.5e-3
 *     rows parallel to 1e-2; to 1e-3                      up to 1.8e-3; 2.6e-3
 *     half of the singular values at 1, half at 1e-2      2.1e-3 to 3.5e-3
 *     an eighth at 1, the others at 1e-3                  2.0e-3 to 3.6e-3
 *     equal rows; equal elements                          up to 5.3e-3; 8.9e-3
 *     rank four; one   65 rows up to 4.6e-3; 9.2e-3, 128 2.8e-3; 4.1e-3, 1000 1.7e-3
 *     all of it in a few rows of the shorter side, of rank one or parallel to
 *     1e-3             2 to 4 rows up to 4.5e-2, 8 3.7e-2, 16 3e-2, 64 9e-3
 *                      parallel to 1e-2: 2 rows up to 1.3e-2, 4 5e-3, 64 1.8e-3
 *
 * (up to: the largest that matrices of 65 to 1500 rows gave, a few of each kind
 * and size).  The scales bound the
 * iterates: the singular values of X have to stay below 4 and those of B below
 * 16 (the default coefficients keep them below 1.3 and 3); beyond, elements
 * overflow to infinity.
 */
#ifndef TG_ORTHO_H
#define TG_ORTHO_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TG_NS_MAX_STEPS 32

/* tg_newton_schulz_workspace_bytes — device memory a call needs as workspace
 * (host-only); -1 if the sizes would be refused. */
int64_t tg_newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);

/*
 * tg_newton_schulz_f32, _f16, _bf16 — enqueue the iteration on fp32, binary16 or
 * bfloat16 matrices.
 *
 *   G         device pointer; element (m, i, j) at G + m·g_stride + i·ldg + j.
 *   O         device pointer to bfloat16, the result, element (m, i, j) at
 *             O + m·o_stride + i·ldo + j.  O may be G itself only where both have
 *             2-byte elements and the same layout.
 *   batch, rows, cols   sizes; nothing happens if one of them is 0.
 *   ldg, ldo  elements between rows, >= cols; g_stride, o_stride elements
 *             between matrices (any value for batch <= 1).
 *   steps     0 to TG_NS_MAX_STEPS (0: the scaled matrix itself).
 *   coefficients  host pointer to 3·steps floats (a, b, c of each step), or NULL
 *             for the default.  Read before the call returns.
 *   eps       added to the norm, >= 0.  A zero matrix gives zeros for eps > 0.
 *   workspace device memory, 256-byte aligned, of at least
 *             tg_newton_schulz_workspace_bytes(batch, rows, cols) bytes; calls
 *             that may overlap must not share one.
 *   stream    hipStream_t.  Only kernels are launched: the call may be recorded
 *             into a graph.
 *
 * A NaN or an infinity in a matrix makes that matrix's result NaN and leaves
 * the others alone.  Repeated calls give the same bits.  Returns TG_OK,
 * TG_ERR_INVALID_ARG (negative sizes, a leading dimension below cols, batches
 * whose o_stride lets results overlap, steps or eps out of range, NULL pointers, a
 * workspace that is NULL, misaligned or too small), TG_ERR_TOO_LARGE (rows or
 * cols >= 2^21 - 64, or 2^23 or more 64×64 blocks in all matrices),
 * TG_ERR_DEVICE or TG_ERR_LAUNCH.
 */
int tg_newton_schulz_f32(const void *G, void *O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                         int64_t g_stride, int64_t ldo, int64_t o_stride, int steps, const float *coefficients,
                         float eps, void *workspace, int64_t workspace_bytes, void *stream);
int tg_newton_schulz_f16(const void *G, void *O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                         int64_t g_stride, int64_t ldo, int64_t o_stride, int steps, const float *coefficients,
                         float eps, void *workspace, int64_t workspace_bytes, void *stream);
int tg_newton_schulz_bf16(const void *G, void *O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                          int64_t g_stride, int64_t ldo, int64_t o_stride, int steps, const float *coefficients,
                          float eps, void *workspace, int64_t workspace_bytes, void *stream);

/* tg_newton_schulz_plan — host-only: the kernels' tile classes for these sizes
 * (truncated to name_len bytes with the NUL); the argument-validation status. */
int tg_newton_schulz_plan(int64_t batch, int64_t rows, int64_t cols, char *name, int64_t name_len);

#ifdef __cplusplus
}
#endif

#endif /* TG_ORTHO_H */
