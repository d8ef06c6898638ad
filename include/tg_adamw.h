/*
 * tg_adamw.h — an AdamW step over many tensors at once, with moments in 32 or
 * in 8 bits (libtg_gemm.so, MI355X / gfx950).
 *
 * For each element p with gradient g, at step t = 1, 2, ...:
 *
 *     g ← s·g                                   (s: the gradients' scale, 1 if none)
 *     m ← β1·m + (1 − β1)·g
 *     v ← β2·v + (1 − β2)·g²
 *     p ← (1 − lr·wd)·p − lr/(1 − β1^t) · m / (√v/√(1 − β2^t) + eps)
 *
 * All of it in fp32, each operation rounded on its own, the quotient within 2 units
 * in the last place; the factors that depend on t, lr and β alone are computed in 64
 * bits and rounded once (an eps below 2^-126 counts as 0).  p of 16 bits
 * is rounded once when it is stored, to nearest: updates below half a step of p
 * are lost, which is why training keeps p in fp32 and lets the call write the
 * 16-bit copy that the model computes with.
 *
 * Moments in 8 bits.  A tensor is cut into blocks of TG_ADAMW_BLOCK consecutive
 * elements, the last one possibly shorter.  A block of m is held as E4M3 values
 * in units of a fp32 scale, its largest magnitude times 1/448 (a value x as
 * x·(1/largest·448), each operation rounded to nearest); for v its root √v is
 * held, the same way, whose exponents span half of v's.  A rounding is at most
 * 2^-4 of the value (and 2^-10 of the unit below 2^-6 of it); the step itself takes
 * m and √v as they are before they are rounded.  Three rules keep the division safe:
 * a root above zero is held as at least the smallest value above zero (2^-9 units)
 * and 2^-74 (the block's largest, where that is below), whose square is a number of
 * fp32, so that v never reads as zero where it is not; a block whose largest magnitude
 * is below 2^-110 is held as zeros; and a NaN or an infinity in a block makes
 * that block's moments not finite (in 32 bits only the element's).  A moment
 * that moves by less than half a step of its format relative to its block's largest
 * stays where it is; √v, which β2 = 0.999 lets fall by 5e-4 of itself a step, then
 * falls with its block's largest, which the scale holds in fp32.
 */
#ifndef TG_ADAMW_H
#define TG_ADAMW_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TG_ADAMW_BLOCK 256

/* Element types of parameters, gradients and copies. */
enum { TG_ADAMW_F32 = 0, TG_ADAMW_F16 = 1, TG_ADAMW_BF16 = 2 };

/* One tensor: device pointers to n consecutive elements each, at the alignment
 * of an element. */
typedef struct {
    void *p;        /* parameters, read and written */
    const void *g;  /* gradients */
    void *m;        /* first moment: fp32, or E4M3 bytes */
    void *v;        /* second moment: fp32, or E4M3 bytes of its root */
    float *m_scale; /* 8 bits only: ceil(n / TG_ADAMW_BLOCK) scales each */
    float *v_scale;
    void *copy;     /* p rounded to copy_type, written; NULL for none */
    int64_t n;      /* nothing happens for 0 */
} tg_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;           /* t, >= 1 */
    const float *lr_at;     /* device pointer that lr is read from instead, or NULL */
    const int64_t *step_at; /* device pointer that t is read from instead, or NULL (t < 1 counts as 1) */
    const float *g_scale;   /* device pointer to s, or NULL */
    int p_type, g_type;     /* g_type is p_type, or any where p is fp32 */
    int copy_type;          /* TG_ADAMW_F16 or _BF16 (not looked at without copies) */
    int bits;               /* 32 or 8 */
} tg_adamw_config;

/*
 * tg_adamw — enqueue one step over `count` tensors.
 *
 * `tensors` and `config` are host memory, read before the call returns; up to
 * 56 tensors go into one launch.  Only kernels are launched and no workspace
 * is needed: the call may be recorded into a graph, with lr_at and step_at where
 * they have to change between replays (the call does not advance the step).
 * Repeated calls on the same inputs give the same bits.
 *
 * Copies may be given where p is fp32.  Returns TG_OK, TG_ERR_INVALID_ARG
 * (negative sizes, NULL or misaligned pointers, unknown types or bits, a β
 * outside [0, 1), lr, eps or weight_decay negative or not finite, step < 1, or
 * memory that is written and belongs to two tensors or roles, or that is written
 * and read as a gradient, g_scale, lr_at or step_at), TG_ERR_TOO_LARGE
 * (n >= 2^35), TG_ERR_DEVICE or TG_ERR_LAUNCH.
 */
int tg_adamw(const tg_adamw_tensor *tensors, int64_t count, const tg_adamw_config *config, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TG_ADAMW_H */
