/*
 * hgemm_adamw.h — C ABI of the optimizer's step on MI355X (gfx950): what takes
 * the gradients that hg_linear_grad gives to the weights that hg_linear reads.
 *
 *   hg_adamw        one step of AdamW over many tensors, their moments in fp32 or
 *                   as 8-bit checkpoints (hgemm_linear.h)
 *   hg_adamw_check  whether its tensors are valid and apart
 *
 * Conventions as in hgemm_linear.h; the array of tensors is HOST memory, read
 * during the call (the launches hold what they need of it).
 */
#ifndef HGEMM_ADAMW_H
#define HGEMM_ADAMW_H

#include "hgemm_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of elements of a tensor, and of tensors in a call; least eps that is not 0. */
#define HG_ADAMW_MAX_ELEMENTS ((int64_t)1 << 36)
#define HG_ADAMW_MAX_TENSORS (1 << 20)
#define HG_ADAMW_LEAST_EPS 1e-30

/*
 * One tensor: n elements one after the other in each array.
 *
 * param    : HG_F16, HG_BF16 or HG_F32, read and written; with a master only
 *            written, the rounded master.
 * master   : the weight in fp32, read and written, or NULL (with HG_F32 it must be).
 * grad     : HG_F16, HG_BF16 or HG_F32.
 * m, v     : the moments, read and written, both of state_type: n fp32 values
 *            (HG_F32), or n codes with ceil(n / 32) scale bytes each (HG_E4M3: the
 *            8-bit checkpoint of bf16 values of a matrix of one row).  Zeros all
 *            through (codes and bytes) are moments of zero.
 */
typedef struct hg_adamw_tensor {
    void *param;
    float *master;
    const void *grad;
    void *m;
    uint8_t *m_scales;
    void *v;
    uint8_t *v_scales;
    int64_t n;
    int32_t param_type, grad_type, state_type;
} hg_adamw_tensor;

/*
 * hg_adamw — with t the step's number, 1 the first, and g the gradient:
 *
 *     m = beta1·m + (1 - beta1)·g,  v = beta2·v + (1 - beta2)·g²
 *     w = w - lr·(decay·w + (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps))
 *
 *  1 count       : tensors, 0 .. HG_ADAMW_MAX_TENSORS.
 *  2 tensors     : HOST array; no array of a tensor may overlap one that is
 *                  written.  Across tensors this call does not look: see
 *                  hg_adamw_check.
 *  3 step        : t >= 1; not used with device_step.
 *  4 device_step : DEVICE value of t, for calls that are captured, or NULL.  Below
 *                  1 nothing is changed (a step that is to be left out).
 *  5 lr, 9 decay : finite, not negative.
 *  6, 7          : beta1, beta2 in [0, 1).
 *  8 eps         : 0, or HG_ADAMW_LEAST_EPS to 1 / HG_ADAMW_LEAST_EPS.
 * 10 factors     : two DEVICE fp32 values, or NULL: what lr and every gradient are
 *                  multiplied by (a schedule; clipping, a loss scale).
 * 11 seed        : of the random rounding of 8-bit moments; a call's with the same
 *                  seed and t rounds alike.
 * 12 stream      : hipStream_t.
 *
 * All in fp32: products and sums of the moments each rounded by itself, the
 * weight's change as it comes, the param's type rounded once to nearest even.
 *
 * 8-bit moments are rounded at random.  Beta2 is near 1, so a step changes v by
 * less than half a code's distance; rounded to nearest it would never change.  A
 * moment goes up or down to one of its two nearest codes, up with the probability
 * of its distance from the lower one (in steps of 2^-16), so that what is lost or
 * gained in a step is zero on average.  The scale is that of hg_checkpoint8_write
 * for bf16 (the smallest that saturates nothing).  A v above 0 never becomes 0
 * (that would make the next step's quotient as large as eps lets it): its least
 * code is 2^-9 of the scale, 2^-18 of the block's largest.  The random bits are 32
 * of a hash of seed, t, the tensor's place in the call and the element's in the
 * tensor, the low 16 for m, the high 16 for v:
 *
 *     mix(x): x ^= x >> 16; x *= 0x9E3779B9; x ^= x >> 15; x *= 0xB504F333; x ^= x >> 16
 *     key = 0; for w in place, t mod 2^32, t / 2^32, seed mod 2^32, seed / 2^32, element / 2^32:
 *         key = mix(key + w + 0x9E3779B9)
 *     bits = mix(element mod 2^32 ^ key)
 *
 * An infinite or NaN gradient makes its element's weight NaN and no other's; its
 * moments are infinite or NaN then, as the sums say (8 bits: NaN).  A finite one
 * whose square passes fp32's range (above 1.8e19, after factors) makes v
 * infinite: with fp32 moments its weight decays and nothing else from that step
 * on, with 8-bit ones v is NaN and so is the next step's weight.
 */
int hg_adamw(int64_t count, const hg_adamw_tensor *tensors, int64_t step, const int64_t *device_step, double lr,
             double beta1, double beta2, double eps, double decay, const float *factors, uint64_t seed, void *stream);

/* hg_adamw_check — 0 if hg_adamw takes these tensors and no array that is
 * written overlaps another, of whichever tensor; -1 or -2 (host only, n·log n of
 * the arrays: once for the tensors of a program, not for every step). */
int hg_adamw_check(int64_t count, const hg_adamw_tensor *tensors);

#ifdef __cplusplus
}
#endif

#endif /* HGEMM_ADAMW_H */
