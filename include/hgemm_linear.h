/*
 * hgemm_linear.h — C ABI of the linear layer on MI355X (gfx950): the product
 * of hgemm.h with the layer's epilogue, its gradient, and the 8-bit
 * checkpoints that keep activations between the two.
 *
 *   hg_linear             z = X·Wᵀ + bias,  Y = act(z) + R, and z saved in 16
 *                         or 8 bits if wanted, in one launch (a second one
 *                         where the sum is cut into slices)
 *   hg_linear_grad        dz = dY·act'(z),  dX = dz·W,  dW = dzᵀ·X,
 *                         dbias = the column sums of dz
 *   hg_checkpoint8_write  a 16-bit matrix as e4m3 codes with one power-of-two
 *   hg_checkpoint8_read   scale for every 32 columns of a row, and back
 *
 * Conventions as in hgemm.h: DEVICE pointers on the current HIP device, calls
 * asynchronous on `stream`, no allocation, no host state, a status that is 0,
 * -i for an invalid argument i (1-based, nothing launched; the first one in
 * the order of the prototype) or 1000 + hipError_t.  The caller owns every
 * buffer; calls from several host threads are safe, and calls that overlap in
 * time need workspaces of their own (so do two captured graphs that may).
 * Every launch may be captured into a HIP graph.
 *
 * Overlap is judged by the bytes from a matrix's first element to its last,
 * except between matrices whose rows are the same number of bytes apart:
 * different columns of one array do not overlap.
 */
#ifndef HGEMM_LINEAR_H
#define HGEMM_LINEAR_H

#include "hgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a matrix next to HG_F16, HG_F32 and HG_BF16: an 8-bit
 * checkpoint (see hg_checkpoint8_write). */
#define HG_E4M3 3

/* Activations next to HG_ACT_NONE and HG_ACT_RELU.  act and act' are computed
 * in fp32 (absolute error of the normal distribution function in GELU:
 * 1.5e-7); at ±inf they take their limits, NaN stays NaN, and ReLU's slope at
 * 0 is 0. */
#define HG_ACT_GELU 2       /* z·Phi(z), Phi the normal distribution function */
#define HG_ACT_GELU_TANH 3  /* z/2·(1 + tanh(sqrt(2/pi)·(z + 0.044715·z³))) */
#define HG_ACT_SILU 4       /* z/(1 + exp(-z)) */

/* Columns that share a scale in an 8-bit checkpoint. */
#define HG_E4M3_BLOCK 32

/* Largest sizes: N and K, M, and any leading dimension. */
#define HG_LINEAR_MAX_WIDTH (1 << 20)
#define HG_LINEAR_MAX_ROWS (1 << 30)
#define HG_LINEAR_MAX_LD (1 << 30)

/*
 * A row-major matrix: element (i, j) at data[i*ld + j], ld >= max(1, columns).
 * Elements behind the last column are neither used nor written.
 * HG_E4M3: data holds one code per element, scales the scale bytes, block b of
 * row i at scales[i*lds + b], lds >= ceil(columns / 32).  scales and lds are
 * ignored for the other types.
 */
typedef struct hg_matrix {
    void *data;
    int64_t ld;
    uint8_t *scales;
    int64_t lds;
    int32_t type;
} hg_matrix;

/*
 * hg_linear — Y = act(X·Wᵀ + bias) + R.
 *
 *  1 act         : HG_ACT_NONE .. HG_ACT_SILU.
 *  2 M, 3 N, 4 K : rows of X, rows of W (columns of Y), length of the sum.
 *  5 X           : M×K, HG_F16 or HG_BF16.
 *  6 W           : N×K, X's type (hgemm's B, K-contiguous).
 *  7 bias        : N fp32 values, or NULL.
 *  8 R           : M×N residual of Y's type, or NULL.  May be Y itself (same
 *                  data and ld): Y is then read and written in place.
 *  9 Y           : M×N, X's type or HG_F32.
 * 10 Z           : M×N, where the pre-activation z = X·Wᵀ + bias is saved, X's
 *                  type or HG_E4M3; NULL: not saved.
 * 11 work        : device workspace, 16-byte aligned, of at least
 * 12 work_bytes    hg_linear_workspace_size(M, N, K, X, W) bytes (often 0).
 * 13 stream      : hipStream_t.
 *
 * Per element, in fp32: the sum of the products (exact in fp32, added in an
 * unspecified but fixed order), + bias, Z rounded from that, act on the
 * unrounded value, + R, and Y rounded once to nearest even.  The result
 * depends only on the arguments (no atomics).  K = 0 sums nothing.  M = 0 or
 * N = 0 touches nothing.
 * No output may overlap an input, another output or the workspace, R = Y
 * excepted (-9, -10, -11).
 * An operand that is not 16-byte aligned, or whose ld or K is no multiple of
 * 8, is first copied to aligned rows in the workspace if the product is large.
 */
int hg_linear(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, const float *bias,
              const hg_matrix *R, const hg_matrix *Y, const hg_matrix *Z, void *work, int64_t work_bytes, void *stream);

/* hg_linear_workspace_size — bytes hg_linear needs for these operands on the
 * current device, whatever Y and Z (host only; of X and W the address'
 * alignment, ld and type are looked at); -i for an invalid argument i. */
int64_t hg_linear_workspace_size(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W);

/*
 * hg_linear_grad — the gradients of hg_linear's X, W and bias.  (R's is dY
 * itself.)
 *
 *  1 act         : the forward call's.
 *  2 M, 3 N, 4 K : the forward call's.
 *  5 dY          : M×N, HG_F16 or HG_BF16.
 *  6 W           : N×K, dY's type; read only for dX (else may be NULL).
 *  7 X           : M×K, dY's type or HG_E4M3; read only for dW (else may be
 *                  NULL).
 *  8 Z           : M×N, the saved pre-activation, dY's type or HG_E4M3; not
 *                  read with HG_ACT_NONE (then may be NULL).
 *  9 dX          : M×K, dY's type, written; NULL: not wanted.
 * 10 dW          : N×K, dY's type or HG_F32; NULL: not wanted.
 * 11 dbias       : N fp32 values; NULL: not wanted.
 * 12 accumulate  : 0: dW and dbias are written; 1: they are added to (in
 *                  fp32, rounded once to dW's type).
 * 13 work        : device workspace, 16-byte aligned, of at least
 * 14 work_bytes    hg_linear_grad_workspace_size(M, N, K, dY, W, X) bytes.
 * 15 stream      : hipStream_t.
 *
 * dz = dY·act'(z) is computed in fp32; dbias sums it unrounded; for the two
 * products it is rounded once to dY's type (their matrix-core operand), so a
 * term of dX or dW carries a relative error of half a step of that type.
 * HG_F16: a dz past 65504 is infinite there, as any value rounded to that type
 * (the slopes of GELU and SiLU reach 1.13 and 1.10, so a dY above 58 000 may
 * give one); dbias stays finite.
 * The sums are fp32, in a fixed order.  M = 0 sums nothing (dW and dbias are
 * zero, or stay as they are), N = 0 gives dX = 0.  No output may overlap an
 * input, another output or the workspace (-9, -10, -11, -13).
 */
int hg_linear_grad(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *dY, const hg_matrix *W,
                   const hg_matrix *X, const hg_matrix *Z, const hg_matrix *dX, const hg_matrix *dW, float *dbias,
                   int accumulate, void *work, int64_t work_bytes, void *stream);

/* hg_linear_grad_workspace_size — bytes hg_linear_grad needs for these
 * operands on the current device, whatever act, Z and the gradients wanted
 * (host only; W or X NULL: its gradient's product is not planned for); -i for
 * an invalid argument i. */
int64_t hg_linear_grad_workspace_size(int64_t M, int64_t N, int64_t K, const hg_matrix *dY, const hg_matrix *W,
                                      const hg_matrix *X);

/*
 * hg_checkpoint8_write — an activation in 8 bits.
 *
 *  1 M, 2 N      : rows and columns, M <= HG_LINEAR_MAX_ROWS, N <=
 *                  HG_LINEAR_MAX_WIDTH.
 *  3 X           : M×N, HG_F16 or HG_BF16.
 *  4 C           : M×N, HG_E4M3; must not overlap X (-4).
 *  5 stream      : hipStream_t.
 *
 * For every 32 consecutive columns of a row (the last block may be shorter),
 * with amax the largest magnitude of its finite elements: e = the smallest
 * integer with amax <= 448·2^e, at least -15 and at most 8 (HG_F16) or at
 * least -117 (HG_BF16); the scale byte is e + 127, and a code is x·2^-e
 * rounded to the nearest OCP e4m3 value, ties to even.  The scaling is exact,
 * so a value is off by at most half a step of e4m3 (2^-4 of it, or 2^-10·2^e
 * near zero), and what a code stands for is exact in X's type.  With the
 * largest e (8 for HG_F16, 120 for HG_BF16: amax above 7/8 of the type's
 * range) codes stop at ±240, because 256·2^e is past that range.
 * Infinities and NaN become NaN codes and leave the block's scale alone.
 */
int hg_checkpoint8_write(int64_t M, int64_t N, const hg_matrix *X, const hg_matrix *C, void *stream);

/*
 * hg_checkpoint8_read — the values an 8-bit checkpoint stands for.
 *
 *  1 M, 2 N      : as hg_checkpoint8_write.
 *  3 C           : M×N, HG_E4M3.
 *  4 X           : M×N, HG_F16 or HG_BF16; must not overlap C (-4).
 *  5 stream      : hipStream_t.
 *
 * code·2^(byte - 127), rounded to nearest even where X's type does not hold it
 * (never for what hg_checkpoint8_write wrote from the same type); a scale byte
 * of 255 stands for NaN.
 */
int hg_checkpoint8_read(int64_t M, int64_t N, const hg_matrix *C, const hg_matrix *X, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HGEMM_LINEAR_H */
