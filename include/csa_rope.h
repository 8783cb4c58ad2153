/*
 * csa_rope.h -- C ABI of the rotary positions of compressed rows, queries and
 * keys (part of libcsa_compress.so).
 *
 * Every head's columns [offset, offset + rope_dim) are rope_dim / 2 pairs
 * (a, b); pair i of a token at position p is turned by the angle p * freqs[i]
 * and scaled by `amplitude`:
 *
 *   a' = amplitude * (a cos - b sin)      b' = amplitude * (b cos + a sin)
 *
 * The other columns are copied. With `transpose` the matrix above is
 * transposed (the angle is negated, the amplitude stays): the gradient with
 * respect to x of a call without it, and for amplitude 1 the inverse turn.
 *
 * Pairs: CSA_ROPE_INTERLEAVED pairs the columns 2i and 2i + 1 of the turned
 * part, CSA_ROPE_HALF the columns i and i + rope_dim / 2.
 *
 * Positions: `positions` [tokens] (int32 or int64, any value, negative ones
 * included) or, when it is null, those of compressed rows: row t of segment s
 * (cu_rows[s] <= t < cu_rows[s + 1]) has the position (t - cu_rows[s]) * ratio,
 * the first token of its block; rows t >= cu_rows[num_seqs] (padding up to a
 * static capacity) have position 0.
 *
 * Angles: frequencies are radians a position in fp64. The kernel holds them
 * in turns as 64-bit fixed-point numbers, within 2^-64 + |freqs[i]| 2^-61 / (2 pi)
 * turns, and multiplies them by the position modulo 2^64: that product and its
 * reduction to one turn are exact. The angle used is within
 *
 *   |p| (2^-64 + |freqs[i]| 2^-61 / (2 pi)) + 2^-33 turns
 *
 * of p * freqs[i]: below 2^-31 for |freqs[i]| <= 1 and |p| <= 2^31, below 2^-12 for
 * |freqs[i]| = 2^20 there (and then rounded to fp32 in half turns, |angle| <= 1:
 * 2^-25). Frequencies must be finite and below 2^62 in magnitude; where the
 * bound passes half a turn, the angle says nothing. Products and sums are fp32,
 * rounded once to the tensor's type.
 *
 * x and y are [tokens, heads, head_dim], the last dimension contiguous, the
 * other two with strides in elements. Input strides may be 0 (a broadcast
 * gradient); the output's elements must be distinct. y == x with the same
 * strides turns in place (columns outside the part are neither read nor
 * written); any other overlap of x and y is not allowed.
 *
 * One kernel launch, asynchronous on `stream`, no host synchronisation, no
 * device memory allocated. tokens == 0 launches nothing.
 */
#ifndef CSA_ROPE_H
#define CSA_ROPE_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "csa_compress.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators beside the Compressor. */
#define CSA_BF16 0
#define CSA_FP16 1
#define CSA_FP32 2

#define CSA_ROPE_INTERLEAVED 0
#define CSA_ROPE_HALF 1

/*
 * Checked on the host (nothing is launched otherwise): dtype and layout
 * known, position_bits 32 or 64 where positions are given, rope_dim even,
 * 2 <= rope_dim, 0 <= offset, offset + rope_dim <= head_dim (UNSUPPORTED);
 * sizes non-negative, heads >= 1, strides >= 0, output elements distinct,
 * ratio >= 1 and num_seqs >= 1 with cu_rows (RANGE); x, y, freqs and one of
 * positions / cu_rows given (NULL); pointers aligned to their element
 * (ALIGN). Any alignment and any sizes within that work; 16-byte aligned
 * rows and parts take the vector kernel.
 */
csa_status_t csa_rope(const void* x, void* y, const double* freqs, const void* positions,
                      int32_t position_bits, const int32_t* cu_rows, int32_t num_seqs,
                      int32_t ratio, int64_t tokens, int32_t heads, int32_t head_dim,
                      int64_t x_token_stride, int64_t x_head_stride, int64_t y_token_stride,
                      int64_t y_head_stride, int32_t rope_dim, int32_t offset, int32_t layout,
                      int32_t dtype, float amplitude, int32_t transpose, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA_ROPE_H */
