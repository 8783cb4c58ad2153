/*
 * csa_norm_rope.h -- C ABI of the norms of queries and keys for each head with
 * the rotary positions in the same pass, and of its gradient (part of
 * libcsa_compress.so).
 *
 * Every head x of a token is normed over its head_dim columns and turned:
 *
 *   r = 1 / sqrt(mean(x^2) + eps)      n_c = x_c r w_c      y = R(p) n
 *
 * with a weight w for each column (of all heads of a side) and R(p) the turn
 * of include/csa_rope.h: the columns [offset, offset + rope_dim) in pairs, by
 * position * freqs, amplitude included, positions given or those of
 * compressed rows. Two sides, queries and keys, go through one launch; the
 * second may be absent. A head of compressed rows is a side as well.
 *
 * The gradient, for g with respect to y:
 *
 *   h = R(p)^T g     dw_c = sum over tokens and heads of h_c x_c r
 *   u = h w          dx_c = r (u_c - x_c r^2 mean(u x))
 *
 * r is worked out again from x. Products, sums and r are fp32, rounded once to
 * the tensor's type. dw is summed in an order that depends on the sizes alone:
 * results are the same from call to call.
 *
 * Tensors are [tokens, heads, head_dim], the last dimension contiguous, the
 * other two with strides in elements. Strides of x and grad may be 0; elements
 * of an output (y, dx) must be distinct. y == x with the same strides works in
 * place, as does dx == x or dx == grad; any other overlap is not allowed.
 *
 * Asynchronous on `stream`, no host synchronisation. One launch forward, two
 * backward with a workspace of the library's stream-ordered pool. With
 * tokens == 0 the forward launches nothing and the backward writes zeros to dw.
 */
#ifndef CSA_NORM_ROPE_H
#define CSA_NORM_ROPE_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "csa_compress.h"
#include "csa_rope.h" /* CSA_BF16 .., CSA_ROPE_INTERLEAVED .. */

#ifdef __cplusplus
extern "C" {
#endif

/* A side. Forward: x, weight, y. Backward: x, weight, grad, y as dx, dweight. */
typedef struct csa_norm_side {
  const void* x;
  const void* weight; /* [head_dim], contiguous, in weight_dtype */
  const void* grad;
  void* y;
  void* dweight; /* [head_dim], contiguous, in weight_dtype */
  int64_t x_token_stride, x_head_stride;
  int64_t grad_token_stride, grad_head_stride;
  int64_t y_token_stride, y_head_stride;
  int32_t heads;
} csa_norm_side_t;

/* What both sides share. */
typedef struct csa_norm_rope {
  const double* freqs;   /* [rope_dim / 2], radians a position, as in csa_rope */
  const void* positions; /* [tokens] int32 or int64, or null: compressed rows  */
  const int32_t* cu_rows;
  int64_t tokens;
  int32_t position_bits, num_seqs, ratio;
  int32_t head_dim, rope_dim, offset;
  int32_t layout;       /* CSA_ROPE_INTERLEAVED, CSA_ROPE_HALF */
  int32_t dtype;        /* of x, y, grad: CSA_BF16, CSA_FP16, CSA_FP32 */
  int32_t weight_dtype; /* dtype or CSA_FP32 */
  float amplitude, eps;
} csa_norm_rope_t;

/*
 * Checked on the host (nothing is launched otherwise), as in csa_rope: types and
 * layout known, 2 <= rope_dim even, the part inside head_dim <= 1024
 * (UNSUPPORTED); sizes, strides, eps >= 0 and finite, distinct output elements
 * (RANGE); null pointers (NULL); pointers aligned to their element (ALIGN).
 * 16-byte aligned rows and parts take the vector kernel (head_dim <= 512 in fp32).
 * k may be null.
 */
csa_status_t csa_norm_rope(const csa_norm_rope_t* how, const csa_norm_side_t* q,
                           const csa_norm_side_t* k, cudaStream_t stream);
csa_status_t csa_norm_rope_bwd(const csa_norm_rope_t* how, const csa_norm_side_t* q,
                               const csa_norm_side_t* k, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA_NORM_ROPE_H */
