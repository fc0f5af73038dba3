/*
 * hgemm_adapters.h — C ABI of the linear layer with low-rank adapters on MI355X
 * (gfx950): the product of hgemm_linear.h for the rows of many requests at
 * once, each with the adapter that its request brings.
 *
 *   hg_linear_adapters    z = X·Wᵀ + bias + s_g·(X·A_gᵀ)·B_gᵀ,  g = which[row],
 *                         Y = act(z) + R, and z saved in 16 or 8 bits if wanted
 *
 * Conventions as in hgemm_linear.h.  Two launches (three or four where hg_linear
 * takes two or three): X·A_gᵀ, then the layer's product, whose kernels add the
 * second half to their sums before anything is rounded.  One row with adapters
 * of a small rank takes one launch.
 *
 * There is no backward entry point.  An adapter is trained with the layer's: T =
 * X·Aᵀ and T·Bᵀ are two hg_linear calls on the rows that have it, their gradients
 * two of hg_linear_grad (dB and dT = dz·B, then dA and dT·A, with dz times s_g as
 * their dY).  What is the caller's then: rows of several adapters are taken apart
 * first, and dX is the sum of two matrices of X's type, each rounded, dz·W (a third
 * hg_linear_grad) and the adapters' dT·A.
 */
#ifndef HGEMM_ADAPTERS_H
#define HGEMM_ADAPTERS_H

#include "hgemm_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest rank, number of adapters, and elements from one to the next. */
#define HG_ADAPTERS_MAX_RANK 256
#define HG_ADAPTERS_MAX_COUNT (1 << 20)
#define HG_ADAPTERS_MAX_STRIDE ((int64_t)1 << 40)

/*
 * Adapters of one rank (pad shorter ones with zeros; ranks that are a multiple of
 * 8 are fastest).  Adapter g: A_g rank×K at A + g·stride_a elements, rows lda
 * apart; B_g N×rank at B + g·stride_b, rows ldb apart (any alignment of 2 bytes;
 * multiples of 8 elements are fastest).
 */
typedef struct hg_adapters {
    const int64_t *which; /* M values: row i's adapter; outside 0 .. count-1: none */
    const float *scales;  /* count values s_g, or NULL: 1 */
    const void *A;
    int64_t lda, stride_a;
    const void *B;
    int64_t ldb, stride_b;
    int64_t count;
    int32_t rank;
    int32_t type; /* of A and B: X's */
} hg_adapters;

/*
 * hg_linear_adapters — arguments 1 to 10 and the result as hg_linear's.
 *
 * 11 adapters    : see above; none of its arrays may overlap Y, Z or the
 *                  workspace.  count = 0 or rank = 0: hg_linear itself.
 * 12 work        : device workspace, 16-byte aligned, of at least
 * 13 work_bytes    hg_linear_adapters_workspace_size(M, N, K, rank, X, W) bytes.
 * 14 stream      : hipStream_t.
 *
 * X·A_gᵀ and its scaling are computed in fp32.  For the second product it is
 * kept in fp32 (few rows), as the sum of three HG_BF16 numbers if Y is HG_F32
 * (all of its 24 bits), or of two numbers of X's type, off by at most 2^-16
 * (HG_BF16) or 2^-22 (HG_F16, and 2^-25 where that is more) of it.  In HG_F16 a
 * value that rounds past 65504 is kept in fp32 in any case (which takes longer in
 * the rows that have one).  Rows whose adapter's B_g holds an infinity or NaN may
 * come out NaN in any column.  Nothing of another row enters a row's result (its
 * last bits may differ with the rows beside it, which choose the order of its
 * sums): what is not finite in one request's row or adapter stays in that
 * request's rows.
 */
int hg_linear_adapters(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W,
                       const float *bias, const hg_matrix *R, const hg_matrix *Y, const hg_matrix *Z,
                       const hg_adapters *adapters, void *work, int64_t work_bytes, void *stream);

/* hg_linear_adapters_workspace_size — bytes hg_linear_adapters needs for these
 * operands on the current device (host only; of X and W the address' alignment,
 * ld and type are looked at); -i for an invalid argument i. */
int64_t hg_linear_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t rank, const hg_matrix *X,
                                          const hg_matrix *W);

#ifdef __cplusplus
}
#endif

#endif /* HGEMM_ADAPTERS_H */
