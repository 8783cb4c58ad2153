/*
 * csa_prompt.h -- C ABI of causal attention over packed sequences (prompts,
 * chunks of them, single tokens over held keys) and of its gradient (part of
 * libcsa_compress.so).
 *
 * Sequence s has the query tokens cu_q[s] .. cu_q[s + 1] - 1 of q and the keys
 * and values cu_k[s] .. cu_k[s + 1] - 1 of k and v (cu_k null: cu_q). With n
 * queries and m keys, the queries are the last n of the m tokens: query i sees
 * the keys
 *
 *   max(0, m - n + i + 1 - window) .. m - n + i      (window 0: from key 0 on)
 *
 * Query head h reads key and value head h / (heads / kv_heads):
 *
 *   z_j = sm_scale * (q . k_j)    out = sum_j softmax(z)_j v_j
 *   lse = log sum_j exp(z_j)
 *
 * A query that sees no key (m < n), or whose logits are all -inf, gets out 0
 * and lse -inf. lse lets the result be merged with attention over other rows
 * (csa_cache_attend over compressed ones, say). Keys that a query does not see
 * take no part in its sums, whatever they hold (NaN and infinities included).
 * A key that it sees with a logit of -inf has weight 0, in the gradient too (but in
 * infinite columns of such a key dq may be NaN, in those of such a query dk: 0 times
 * infinity). Where grad is not
 * finite, the gradients of the keys that its query sees are not either.
 *
 * The gradient, for grad with respect to out and grad_lse to lse:
 *
 *   delta = sum_c grad_c out_c - grad_lse      P = exp(z - lse)
 *   dS = P (grad . v - delta)                  dv = P^T grad
 *   dq = sm_scale dS k                         dk = sm_scale dS^T q
 *
 * dk and dv of a key head are summed over its query heads. A query that sees one
 * key has dS = -P delta' with delta' = -grad_lse, exactly.
 *
 * q, k, v and grad are [tokens, heads, head_dim], bf16 or fp16, the last
 * dimension contiguous, the other two with strides in elements (multiples of
 * 8, above 0 where stepped); views of one projection's output work. out, rest, dq,
 * dk, dv ([tokens, heads, head_dim]) and lse, grad_lse ([tokens, heads], fp32) are
 * contiguous. Outputs overlap no input.
 *
 * Logits, softmax statistics and sums are fp32. The tensor core's sums truncate: a
 * row's over n keys lose up to n 2^-28 of their size, 2^-11 for 131072 keys; dk and
 * dv, sums over all queries of up to 128 heads, are taken in parts that lose no more
 * than 2^-12. The weights P and dS enter the second products in the inputs' type;
 * fp16 lifts dS by one power of two for the whole call, which the largest finite rows
 * of grad, grad_lse and v allow. rest (may be null) is what the rounding of out left
 * off, out + rest being exact to twice the bits: with it the gradient's delta loses
 * nothing to that rounding.
 *
 * Rows of no sequence (before cu_q[0], at or behind cu_q[num_seqs]) are left as
 * they were, or with CSA_FILL_OUT become 0 in out and rest, with CSA_FILL_LSE
 * -inf in lse; their dq, and dk and dv of such keys, are 0. cu_q and cu_k do not
 * decrease and end within the tensors. The queries of a sequence that passes a
 * tensor's end see no key: out 0, lse -inf, and gradients of 0 for its rows. With
 * lists that decrease it is not specified what rows hold. Kernels stay inside the
 * buffers whatever the lists hold.
 *
 * Asynchronous on `stream`, no host synchronisation; lengths are read on the
 * device. Workspaces come from the library's stream-ordered pool. Results are the
 * same from call to call. Waits inside the kernels are bounded: rows whose work did
 * not go on for more than a second become NaN.
 */
#ifndef CSA_PROMPT_H
#define CSA_PROMPT_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "csa_compress.h"
#include "csa_rope.h" /* CSA_BF16, CSA_FP16 */

#ifdef __cplusplus
extern "C" {
#endif

typedef struct csa_prompt {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* cu_q; /* [num_seqs + 1] */
  const int32_t* cu_k; /* [num_seqs + 1] or null */
  int64_t num_q, num_k; /* tokens of q, of k and v */
  int64_t q_token_stride, q_head_stride;
  int64_t k_token_stride, k_head_stride;
  int64_t v_token_stride, v_head_stride;
  int32_t num_seqs, heads, kv_heads, head_dim;
  int32_t dtype;  /* CSA_BF16, CSA_FP16 */
  int32_t window; /* tokens that a query sees, its own included; 0: all */
  float sm_scale;
} csa_prompt_t;

#define CSA_FILL_OUT 1
#define CSA_FILL_LSE 2

/*
 * Envelope: head_dim a multiple of 8 up to 128, heads a multiple of kv_heads, at
 * most 128 of them a key head, at most 65535 key heads (UNSUPPORTED); sm_scale positive and
 * finite, tokens < 2^31, tokens * heads < 2^31, num_seqs <= 262144, strides
 * (RANGE); 16-byte aligned tensors (ALIGN). out or lse may not be null, rest may.
 * num_q == 0 launches nothing.
 */
csa_status_t csa_prompt_attend(const csa_prompt_t* p, void* out, void* rest, float* lse,
                               int32_t fill, cudaStream_t stream);

/*
 * out, rest (may be null) and lse are the forward's. grad_lse may be null. dq, dk
 * and dv are written in full.
 */
csa_status_t csa_prompt_attend_bwd(const csa_prompt_t* p, const void* out, const void* rest,
                                   const float* lse, const void* grad, int64_t grad_token_stride,
                                   int64_t grad_head_stride, const float* grad_lse, void* dq,
                                   void* dk, void* dv, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA_PROMPT_H */
