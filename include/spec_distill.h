/*
 * spec_distill.h -- C ABI of distillation from a teacher's top logits, forward
 * and backward, on AMD Instinct MI355X (gfx950).
 *
 * The operation: a draft model is worth what the verifier accepts of it, and
 * acceptance is 1 - TV(p, q) (see spec_verify.h): a draft is trained towards
 * the target's distribution. Of the target only the top entries of each row
 * are kept (a top-k of its logits); the loss is the Kullback-Leibler divergence
 * of the draft's row from that list.
 * The lists of spec_verify_outcomes hold probabilities, not logits, and for
 * every length below G those of the residual max(0, p - q), which is no teacher
 * for the draft. The list of length G is the target's own row: its tokens are
 * the ids, the logarithms of its probabilities the teacher logits, with
 * teacher_lse 0 (they are normalised over the whole vocabulary) and temperature
 * 1 (or T times the logarithms with temperature T, where the draft's row is
 * scaled by T as well).
 *
 * Precise definition, per row n with T = temperature[n], r = fl32(1/T):
 *   x_v = fl32(z[n][v] * r)              the draft's (student's) scaled logits
 *   y_j = fl32(teacher[n][j] * r)        the teacher's, for j with ids[n][j] >= 0
 *   lse = log sum_v exp(x_v);
 *   p_j = exp(y_j - lse_t), lse_t = teacher_lse[n] (the teacher's normaliser
 *         over its whole vocabulary, scaled logits: the listed mass P = sum_j
 *         p_j is then below 1) or, with teacher_lse NULL, the normaliser over
 *         the list (P = 1);
 *   loss[n]    = sum_j p_j (log p_j - (x_{ids[j]} - lse));
 *   grad[n][v] = weight[n] * r * (P exp(x_v - lse) - sum_{j: ids[j] = v} p_j),
 *         the derivative of sum_n weight[n] loss[n] with respect to z[n][v].
 * Entries: a negative id marks an unused entry; its teacher logit is not
 * used. An entry with p_j = 0 adds nothing; one with p_j > 0 whose student
 * logit is -inf makes the loss +inf and the gradient still finite. An id may
 * appear more than once (each entry counts).
 * Rows: a row without a used entry, or whose used teacher logits are all -inf
 * and teacher_lse is NULL, has loss 0 and gradient 0 (a padded row; its logits
 * are not looked at and its lse is NaN). Student logits of -inf are allowed
 * (gradient 0 there). A row with an id >= V, with a temperature that is not
 * positive and finite or whose reciprocal overflows, or whose lse is not finite
 * (no finite logit, a NaN or +inf logit) has loss, lse and its whole gradient
 * NaN; so does one whose teacher normaliser or listed mass P is not finite (a
 * NaN or +inf teacher logit).
 * Arithmetic: exponentials of the V student entries in binary32, their sums
 * in binary64 over binary32 sums of one 16-byte load; the list in binary64;
 * loss rounded once to binary32, gradients once to the logits' dtype. lse is
 * within 2^-23 (ln V + 6) of the exact value, plus its own rounding to binary64.
 * Far rows: any finite scaled logits are allowed. A row whose largest one is
 * beyond +-2.9e6 (2^22 / log2 e; a row masked throughout with a large finite
 * constant) is formed in binary64 against that largest logit, which takes one
 * workgroup several passes over the row. So large an lse no longer holds the
 * logarithm of the sum to the bound above, or at all: the backward call takes
 * from it only that the row is far, and forms the sum again from the logits.
 * Rows whose weight * P / T is past binary32's largest value take that way too
 * (entries that are finite then stay so).
 *
 * Layouts: dense row-major DEVICE arrays owned by the caller: logits, grad
 * [N, V] (SPEC_BF16 or SPEC_F32, aligned to the element, any V), ids [N, K]
 * int32, teacher [N, K] float32, teacher_lse [N] float64 or NULL, temperature,
 * weight, loss [N] float32, lse [N] float64. grad may be the logits array
 * itself (the gradient then takes its place); no other overlap. 1 <= K <=
 * SPEC_DISTILL_MAX_K, V >= 1, 0 <= N < 2^22 (one dispatch).
 *
 * Asynchrony and errors: as in spec_verify.h; each call enqueues one kernel on
 * hip_stream (a hipStream_t, NULL = the null stream), needs no workspace, and
 * may be captured into a HIP graph.
 */
#ifndef SPEC_DISTILL_H
#define SPEC_DISTILL_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest teacher list of a row. */
#define SPEC_DISTILL_MAX_K 256

/* The loss and the row normalisers (which the backward call takes). */
int spec_distill_forward(int rows, int vocab, int dtype, int top_k, const void* logits,
                         const int32_t* ids, const float* teacher, const double* teacher_lse,
                         const float* temperature, float* out_loss, double* out_lse,
                         void* hip_stream);

/* The gradient, from the forward call's inputs and normalisers (or those of
 * spec_lowrank_head for the same logits and temperatures). */
int spec_distill_backward(int rows, int vocab, int dtype, int top_k, const void* logits,
                          const int32_t* ids, const float* teacher, const double* teacher_lse,
                          const float* temperature, const double* lse, const float* weight,
                          void* out_grad, void* hip_stream);

/* Both at once, where the weights are known before the loss is: the logits
 * are read once instead of twice (the first 311 296 bytes of a row, which one
 * workgroup keeps in registers; what is behind them is read again). */
int spec_distill_loss_grad(int rows, int vocab, int dtype, int top_k, const void* logits,
                           const int32_t* ids, const float* teacher, const double* teacher_lse,
                           const float* temperature, const float* weight, float* out_loss,
                           double* out_lse, void* out_grad, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_DISTILL_H */
