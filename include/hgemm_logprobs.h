/*
 * hgemm_logprobs.h — C ABI of what follows a model's last product (hg_linear with
 * the head's weight) on MI355X (gfx950): the distribution over the next token
 * that a row of logits stands for, and the gradient that goes back to
 * hg_linear_grad.
 *
 *   hg_logprobs       log probabilities of given tokens, entropy, the most
 *                     probable tokens with theirs, the softmax's statistics
 *   hg_logprobs_grad  the gradient of log probabilities and entropy
 *
 * Conventions as in hgemm_linear.h.  p = softmax(scale·x) of a row x; all sums
 * are fp32, in an order that depends on M, V and the rows' addresses alone.
 */
#ifndef HGEMM_LOGPROBS_H
#define HGEMM_LOGPROBS_H

#include "hgemm_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of logits in a row, of the most probable tokens, and scale. */
#define HG_LOGPROBS_MAX_VOCABULARY (1 << 20)
#define HG_LOGPROBS_MAX_TOP 32
#define HG_LOGPROBS_MAX_SCALE 1e30f

/*
 * hg_logprobs — one pass over the logits.
 *
 *  1 M           : rows, at most HG_LINEAR_MAX_ROWS.
 *  2 V           : logits in a row, at least 1.
 *  3 X           : M×V, HG_F16, HG_BF16 or HG_F32.
 *  4 scale       : above 0, at most HG_LOGPROBS_MAX_SCALE (1 / temperature).
 *  5 tokens      : M values, or NULL; outside 0 .. V-1: none.
 *  6 logp        : M fp32 values log p[token], 0 where there is none, or NULL
 *                  (with tokens NULL it must be).
 *  7 entropy     : M fp32 values -Σ p·log p, or NULL.
 *  8 stats       : M pairs of fp32 for hg_logprobs_grad, or NULL: the largest
 *                  logit x* and log Σ exp(scale·(x - x*)); the logarithm of the
 *                  softmax's sum is scale·x* + that.
 *  9 top         : 0 .. min(V, HG_LOGPROBS_MAX_TOP).
 * 10 top_ids     : M×top token numbers, the most probable first, of equal
 *                  logits the lower number first; NULL: not wanted.
 * 11 top_logp    : M×top fp32 values, their log probabilities; NULL: not wanted.
 * 12 work        : device workspace, 16-byte aligned, of at least
 * 13 work_bytes    hg_logprobs_workspace_size(M, V, top) bytes (often 0).
 * 14 stream      : hipStream_t.
 *
 * A logit of -inf is a token that cannot be: p = 0, and it adds nothing to the
 * entropy; in a row without any other, log p is -inf, the entropy 0, and stats
 * are (-inf, -inf).  A log probability past fp32's range (a mask of the type's
 * lowest value beside its largest) is -inf.  A NaN or +inf makes the row's log p
 * and entropy NaN; among the most probable tokens a NaN takes the place of a
 * -inf.  The difference of a logit from the largest is formed before it is
 * scaled.
 * No output may overlap an input, another output or the workspace (-6, -7, -8,
 * -10, -11, -12).
 */
int hg_logprobs(int64_t M, int64_t V, const hg_matrix *X, float scale, const int64_t *tokens, float *logp, float *entropy,
                float *stats, int top, int64_t *top_ids, float *top_logp, void *work, int64_t work_bytes, void *stream);

/* hg_logprobs_workspace_size — bytes hg_logprobs needs on the current device
 * (host only); -i for an invalid argument i. */
int64_t hg_logprobs_workspace_size(int64_t M, int64_t V, int top);

/*
 * hg_logprobs_grad — dX = scale·(dlogp·(1[token] - p) - dentropy·p·(log p + entropy)).
 *
 *  1 M, 2 V, 3 X, 4 scale, 5 tokens : the forward call's (tokens may be NULL
 *                  with dlogp NULL).
 *  6 stats       : the forward call's.
 *  7 entropy     : the forward call's; read only for dentropy (else may be NULL).
 *  8 dlogp       : M fp32 values, or NULL: 0; not used in rows without a token.
 *  9 dentropy    : M fp32 values, or NULL: 0.
 * 10 dX          : M×V, X's type, rounded once.  May be X itself (same data and
 *                  ld): the gradient takes the logits' place.
 * 11 stream      : hipStream_t.
 *
 * A row whose logits are all -inf gets zeros.  dX may overlap nothing else
 * (-10).
 */
int hg_logprobs_grad(int64_t M, int64_t V, const hg_matrix *X, float scale, const int64_t *tokens, const float *stats,
                     const float *entropy, const float *dlogp, const float *dentropy, const hg_matrix *dX, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HGEMM_LOGPROBS_H */
