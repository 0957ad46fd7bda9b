/*
 * spec_beam.h -- C ABI of beam selection over beams and vocabulary, and of the
 * reordering of the beams' states, on AMD Instinct MI355X (gfx950).
 *
 * The operation: a draft tree is grown level by level (SpecLA summary,
 * Methodology section 3: tree drafting), each level keeping the `keep` best
 * continuations over all of a sequence's beams and the whole vocabulary; so
 * is a beam search. The selection reads the draft head's logits where they
 * lie and gives what spec_tree.h takes: a node's parent, its token, and its
 * token's log-probability given its path (out_logq). The state each beam
 * carries (recurrent states, key-value prefixes) then has to follow its beam.
 *
 * Precise definition, per sequence b with W = beams, K = keep:
 *   logq(w, v)  = (double)z[b][w][v] - lse[b][w];
 *   value(w, v) = (double)score[b][w] + logq(w, v)       (binary64, two roundings).
 *   Candidates are the pairs (w, v) with a finite logit z, of beams whose score
 *   and normaliser are finite: a score of -inf drops a beam (one that has
 *   ended, or one of a shorter list), a logit of -inf drops a token.
 *   The K first candidates in the order of: larger value; lower w; larger
 *   logit; lower v are kept (within a beam the value never falls with the
 *   logit, so this is the order of value, then of the flat index w * V + v,
 *   except where two different logits of one beam round to one value). Output j holds the j-th: out_parent
 *   = w, out_token = v, out_score = fl32(value), out_logq = fl32(logq). With
 *   fewer than K candidates the rest holds parent -1, token -1, -inf, -inf.
 * lse: the row normalisers in binary64 as spec_lowrank_head returns them for
 * temperature 1 (zeros when the logits are log-probabilities already). NULL:
 * the call forms lse[b][w] = log sum_v exp(z[b][w][v]) itself in the same pass
 * over the logits, exponentials in binary32 and sums in binary64, within
 * 2^-23 (ln V + 6) of the exact value (as a rule a hundred times closer; one
 * beyond +-2^22, of a beam masked with a large finite constant, stays apart as
 * M + log S with M the beam's largest logit, and logq is (z - M) - log S); a
 * beam with a NaN or +inf logit then has no candidates. Two candidates of
 * different beams whose values are closer than that may then come in either
 * order (the same one on every call).
 *
 * Layouts: dense row-major DEVICE arrays owned by the caller: logits [B, W, V]
 * in the context's dtype (aligned to the element; any V), score [B, W]
 * float32, lse [B, W] float64; out_parent, out_token [B, K] int32, out_score,
 * out_logq [B, K] float32 (out_logq may be NULL). out_score may be the score
 * array when K == W; no other overlap.
 *
 * Asynchrony and errors: as in spec_verify.h. spec_beam_select enqueues two
 * kernels on the context's stream and returns; it may be captured into a HIP
 * graph. Calls on one context share its workspace and must not overlap in
 * time, replays of graphs that captured it included. The reordering takes its
 * stream as an argument: give it the context's, or order the two. A context belongs to the
 * device that was current when it was made: SPEC_ESTATE on another one. Its
 * streams have to be that device's.
 */
#ifndef SPEC_BEAM_H
#define SPEC_BEAM_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most beams a selection reads and most candidates it keeps. */
#define SPEC_BEAM_MAX 64

typedef struct spec_beam_ctx spec_beam_ctx;

/* Workspace for selections of this shape (8 bytes per kept candidate of each
 * vocabulary piece of each beam). 1 <= beams, keep <= SPEC_BEAM_MAX, vocab >=
 * 1, batch >= 1; SPEC_EINVAL otherwise or when batch * beams * pieces of the
 * vocabulary would not fit one dispatch. hip_stream may be NULL. */
int spec_beam_init(int batch, int beams, int keep, int vocab, int dtype, void* hip_stream,
                   spec_beam_ctx** out_ctx);

int spec_beam_set_stream(spec_beam_ctx* ctx, void* hip_stream);

int spec_beam_select(spec_beam_ctx* ctx, const void* logits, const float* score,
                     const double* lse, int32_t* out_parent, int32_t* out_token,
                     float* out_score, float* out_logq);

int spec_beam_destroy(spec_beam_ctx* ctx);

/*
 * The states follow their beams: for every layer l, sequence b and slot j,
 *   dst[l][b][j][0 .. bytes) = src[l][b][parent[b][j]][0 .. bytes)
 * where parent[b][j] lies in [0, beams_in); any other parent (-1: no beam)
 * leaves the slot as it is. State (l, b, w) of src starts at byte
 * ((l * batch + b) * beams_in + w) * src_stride, of dst at ((l * batch + b) *
 * beams_out + j) * dst_stride: with a stride larger than `bytes` a prefix of
 * each state is moved and the rest left alone.
 * dst == src with equal strides and beams_in == beams_out reorders in place
 * (also where several slots take one parent); slots that keep their state are
 * then not touched. Otherwise the two ranges must not overlap (SPEC_EINVAL).
 * parent [batch, beams_out] int32 must not lie in either range.
 * 1 <= beams_in, beams_out <= SPEC_BEAM_MAX; layers, batch, bytes >= 0 (0:
 * nothing to do); strides >= bytes. 16-byte accesses are used where pointers,
 * strides and bytes allow them, else 4-byte or single-byte ones. Enqueues one
 * kernel on hip_stream (a hipStream_t, NULL = the null stream).
 */
int spec_beam_reorder(int layers, int batch, int beams_in, int beams_out, const int32_t* parent,
                      const void* src, int64_t src_stride, void* dst, int64_t dst_stride,
                      int64_t bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_BEAM_H */
