/*
 * spec_logprobs.h -- C ABI of the scores of given tokens (log-probability,
 * rank, the row's entropy, top alternatives), and of the gradient of
 * log-probability and entropy, on AMD Instinct MI355X (gfx950).
 *
 * The operation: what a server returns beside the tokens it emits, what a
 * draft's confidence is judged by (the entropy of its rows), what
 * spec_accept_logprobs takes (the tokens' log-probabilities under draft and
 * target), and the list that spec_distill.h calls a teacher, all from one pass
 * over the logits; and its gradient, for a draft trained on tokens
 * (log-likelihood, or a policy's gradient with an entropy bonus).
 *
 * Precise definition, per row n with T = temperature[n], r = fl32(1/T) (no
 * temperatures: r = 1):
 *   x_v = fl32(z[n][v] * r);  M = max_v x_v;  S = sum_v exp(x_v - M);
 *   out_norm[n]    = (M, log S): the row's normaliser is their sum. Apart they
 *                    stay exact where M is far larger than log S (a row masked
 *                    with a large finite constant);
 *   out_logprob[n] = (x_t - M) - log S, t = token[n];
 *   out_rank[n]    = entries before t in the order of larger z, then lower v
 *                    (0: t is the most likely one; -0 and +0 are one logit);
 *   out_entropy[n] = -sum_v p_v log p_v, p_v = exp(x_v - M) / S (0 where p_v = 0);
 *   out_top_token[n], out_top_logprob[n]: the first top_k entries of that order with
 *                    x_v > -inf; the rest of the list is -1, -inf.
 * Tokens: a negative token marks a row without one: logprob 0, rank -1, the
 * other outputs as usual. A token >= V has logprob NaN and rank -1.
 * Rows: entries of -inf are masked. A row with nothing else (every x_v -inf) has
 * norm (-inf, 0), entropy 0, rank -1, an empty list and logprob -inf (0 without
 * a token). A row with a NaN or an x_v of +inf, or whose temperature is not
 * positive and finite or has a reciprocal that overflows, has NaN in every
 * float output, rank -1 and tokens -1.
 * Arithmetic: exponentials in binary32, sums in binary64 over binary32 sums of
 * up to four 16-byte loads, logarithms in binary64; each output rounded once to
 * binary32. log S is within 2^-23 (ln V + 6) of the exact value before that.
 *
 * Backward, with a = grad_logprob[n], b = grad_entropy[n] (NULL: 0):
 *   out_grad[n][v] = r (a ([v = t] - p_v) - b p_v (log p_v + H)),
 * the derivative of sum_n (a logprob + b entropy) with respect to z[n][v]; p
 * and H from norm and entropy, which the forward call returned. a counts as 0
 * in rows without a token. Gradients are 0 at masked entries, whatever a and b,
 * but for the token itself where that is masked (r a, as p_t = 0; its logprob is
 * -inf), 0 in rows with nothing but masked entries, NaN throughout in a row whose
 * scores are NaN (a token >= V included), and rounded once to the logits' dtype.
 *
 * Layouts: dense row-major DEVICE arrays owned by the caller: logits, out_grad
 * [N, V] in the context's dtype (aligned to the element, any V), token, out_rank
 * [N] int32, temperature (or NULL), out_logprob, out_entropy, grad_logprob,
 * grad_entropy (or NULL) [N] float32, out_norm [N, 2] float32, out_top_token [N, K]
 * int32 and out_top_logprob [N, K] float32 (NULL when the context's top_k is
 * 0). out_grad may be the logits array itself (the gradient then takes its
 * place); no other overlap. 0 <= N <= the context's rows.
 *
 * Asynchrony and errors: as in spec_verify.h. The forward call enqueues one or
 * two kernels on the context's stream, the backward call one; both may be
 * captured into a HIP graph. Forward calls on one context share its workspace
 * and must not overlap in time, replays of graphs that captured them included;
 * the backward call uses none. A context belongs to the device that was current
 * when it was made: SPEC_ESTATE on another one. Its streams have to be that
 * device's.
 */
#ifndef SPEC_LOGPROBS_H
#define SPEC_LOGPROBS_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest list of top alternatives. */
#define SPEC_LOGPROBS_MAX_K 64

typedef struct spec_logprobs_ctx spec_logprobs_ctx;

/* Workspace for calls of at most `rows` rows: the parts of rows that several
 * workgroups share. 1 <= rows < 2^24, vocab >= 1, 0 <= top_k <=
 * SPEC_LOGPROBS_MAX_K; SPEC_EINVAL otherwise. hip_stream may be NULL. */
int spec_logprobs_init(int rows, int vocab, int top_k, int dtype, void* hip_stream,
                       spec_logprobs_ctx** out_ctx);

int spec_logprobs_set_stream(spec_logprobs_ctx* ctx, void* hip_stream);

int spec_token_logprobs(spec_logprobs_ctx* ctx, int rows, const void* logits, const int32_t* token,
                        const float* temperature, float* out_logprob, int32_t* out_rank,
                        float* out_entropy, int32_t* out_top_token, float* out_top_logprob,
                        float* out_norm);

int spec_token_logprobs_backward(spec_logprobs_ctx* ctx, int rows, const void* logits,
                                 const int32_t* token, const float* temperature, const float* norm,
                                 const float* entropy, const float* grad_logprob,
                                 const float* grad_entropy, void* out_grad);

int spec_logprobs_destroy(spec_logprobs_ctx* ctx);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGPROBS_H */
