/*
 * spec_int8.h -- C ABI of the draft head's matrix product in 8-bit integers
 * with a scale for each token and channel, and of the quantisation of rows
 * that feeds it, on AMD Instinct MI355X (gfx950).
 *
 * The operation: a draft head's products z = W h (SlimSpec summary,
 * Methodology, architecture: W_up W_down h, or the full head) read all of W
 * for every draft step; 8-bit weights halve those bytes, and integer matrix
 * instructions run at twice the bf16 rate.
 *
 * Quantisation of x [N, D], per row n (a token's activation, or a vocabulary
 * entry's weights):
 *   scale[n] = fl32(max_k |x[n][k]| / 127);
 *   q[n][k]  = x[n][k] / scale[n] rounded to the nearest integer, ties to
 *              even, from the exact quotient, at most 127 in magnitude.
 * A row of zeros (or one whose scale underflows to 0) gets scale 0 and q = 0;
 * a row with a NaN or infinity gets scale NaN and q = 0, so that what is made
 * of it is NaN as well.
 *
 * Product, a [N, D] int8 with a_scale [N], w [V, D] int8 with w_scale [V]:
 *   acc[n][v] = sum_k a[n][k] * w[v][k]                        (int32, exact)
 *   out[n][v] = ((float)acc * a_scale[n]) * w_scale[v]   (binary32), rounded
 *               to bf16 (to nearest even) when out_dtype is SPEC_BF16.
 * Every 8-bit value is allowed, -128 included.
 *
 * Layouts: dense row-major DEVICE arrays owned by the caller. spec_quantize_rows:
 * x in `dtype` (SPEC_F32 or SPEC_BF16, aligned to the element), any D >= 1.
 * spec_int8_product: D % 16 == 0, 16 <= D <= SPEC_INT8_MAX_DEPTH (the sum
 * stays inside int32), a and w 16-byte aligned; out aligned to its element, any
 * V >= 1. N >= 0. Outputs must not overlap inputs. One dispatch limits the
 * sizes: N < 2^24 rows in spec_quantize_rows; in spec_int8_product the tiles of
 * the output, which every output that fits the card's memory stays below (N <
 * 2^31 - 256 for the narrowest). SPEC_EINVAL beyond.
 *
 * Asynchrony and errors: as in spec_verify.h; each call enqueues one kernel on
 * hip_stream (a hipStream_t, NULL = the null stream), needs no workspace, and
 * may be captured into a HIP graph.
 */
#ifndef SPEC_INT8_H
#define SPEC_INT8_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 2^17 - 16: the largest depth with D * 2^14 < 2^31 (products of -128s). */
#define SPEC_INT8_MAX_DEPTH 131056

int spec_quantize_rows(int rows, int cols, int dtype, const void* x, int8_t* out_q,
                       float* out_scale, void* hip_stream);

int spec_int8_product(int rows, int depth, int cols, const int8_t* a, const float* a_scale,
                      const int8_t* w, const float* w_scale, int out_dtype, void* out,
                      void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_INT8_H */
