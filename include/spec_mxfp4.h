/*
 * spec_mxfp4.h -- C ABI of the draft head's matrix product in 4-bit floating
 * point with a scale for every 32 entries (the microscaling format of e2m1
 * elements and E8M0 scales), and of the quantisation of rows that feeds it, on
 * AMD Instinct MI355X (gfx950).
 *
 * The operation: a draft head's products z = W h (SlimSpec summary,
 * Methodology, architecture: W_up W_down h, or the full head) read all of W
 * for every draft step; 4-bit weights are half the bytes of spec_int8.h's, a
 * scale follows every 32 entries instead of a whole row, and the matrix
 * instructions that apply the scales run at four times the bf16 rate.
 *
 * Layout of a quantised row of D entries: D is rounded up to D' =
 * SPEC_MXFP4_PADDED(D), whole groups of 128. D' / 2 bytes of codes, byte j
 * holding entry 2 j in its low and 2 j + 1 in its high half, and D' / 32 scale
 * bytes, byte b for entries 32 b .. 32 b + 31.
 *   code c: sign (c & 8), magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6 for c & 7 = 0 .. 7;
 *   scale byte s: 2^(s - 127); 255 stands for NaN.
 * An entry is its code's value times its scale.
 *
 * Quantisation of x [N, D], for each block of 32 entries (the last may be
 * shorter), A = max |x| over the block:
 *   e = max(floor(log2 A) - 2, -127), of a block of zeros -127; the byte is e + 127;
 *   a code is x / 2^e rounded to the nearest magnitude, ties to the even code,
 *   at most 6 (A / 2^e lies below 8: what is above 6 saturates). x's sign is
 *   kept, that of a zero too.
 * A block with a NaN or infinity gets the byte 255 and codes 0, and all of it
 * stands for NaN. Entries and blocks past D get codes 0 and bytes 0.
 * out_values [N, D] in x's dtype (or NULL) takes what the codes stand for,
 * which both dtypes hold exactly.
 *
 * Product, a [N, D'] with scales, w [V, D'] with scales (written A, S below):
 *   out[n][v] = sum_b 2^(Sa[n][b] + Sw[v][b] - 254) sum_{k in block b} A[n][k] W[v][k]
 * accumulated in binary32 by the matrix instructions, each of which adds two
 * blocks (whose own sums are exact) of either half of a stage of K, and rounded
 * to bf16 (to nearest even) when out_dtype is SPEC_BF16. A NaN block makes every
 * output that reads it NaN. While no partial sum leaves binary32's normal range,
 * the sum is within D' / 64 * 2^-23 of sum_k |A W| 2^(...) of the exact one.
 *
 * Layouts: dense row-major DEVICE arrays owned by the caller. Codes and scales
 * are 16-byte and 4-byte aligned for the product, both 4-byte aligned for the
 * quantisation; x, out_values and out are aligned to their element. Any D >= 1
 * and V >= 1, N >= 0; depth is D'. out_values may be x itself (the values then
 * take its place); no other overlap. Each call is one dispatch: N * D' < 2^35
 * in the quantisation, and in the product at most 2^31 - 4096 tiles of up to 256
 * rows x 256 entries; SPEC_EINVAL beyond.
 *
 * Asynchrony and errors: as in spec_verify.h; each call enqueues one kernel on
 * hip_stream (a hipStream_t, NULL = the null stream), needs no workspace, and
 * may be captured into a HIP graph.
 */
#ifndef SPEC_MXFP4_H
#define SPEC_MXFP4_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Entries that a row of D entries is padded to. */
#define SPEC_MXFP4_PADDED(D) (((D) + 127) / 128 * 128)

/* Largest depth of the product: the sum's bound above is 2^-9 of sum_k |A W| there. (The
 * kernel's addresses would hold to a depth below 2^25.) */
#define SPEC_MXFP4_MAX_DEPTH (1 << 20)

int spec_mxfp4_quantize_rows(int rows, int cols, int dtype, const void* x, uint8_t* out_q,
                             uint8_t* out_scale, void* out_values, void* hip_stream);

int spec_mxfp4_product(int rows, int depth, int cols, const uint8_t* a, const uint8_t* a_scale,
                       const uint8_t* w, const uint8_t* w_scale, int out_dtype, void* out,
                       void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_MXFP4_H */
