// Shared by the translation units of causal attention over packed sequences
// (csa_prompt.cu and its kernels). Not installed, not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_prompt.h"

namespace csa {

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* g;      // grad
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* out;
  void* rest;
  float* lse;
  const float* grad_lse;
  void* dq;
  void* dk;
  void* dv;
  int64_t qt, qh, kt, kh, vt, vh, gt, gh;  // strides in elements
  int32_t num_q, num_k;
  int32_t nseq, heads, kv, group, d, window;
  int32_t fill;
  float scale;
  int32_t polls;  // of a wait, before its CTA gives up
};

// PromptArgs::polls: kPolls (csa_tc.cuh), unless a test has set it lower.
extern "C" int32_t csa_prompt_polls;

// A sequence's rows. Where its lists pass the tensors, or one of them decreases, its queries see
// no key: to a kernel of query rows it has those inside q and no keys, to one of keys (KEYS)
// those inside k and no queries, so that their results are written all the same.
struct Span {
  int32_t q0, nq, k0, nk;
};
template <bool KEYS>
__device__ __forceinline__ Span span_of(const PromptArgs& a, int s) {
  Span w;
  w.q0 = __ldg(a.cu_q + s);
  w.k0 = __ldg(a.cu_k + s);
  const int32_t q1 = __ldg(a.cu_q + s + 1), k1 = __ldg(a.cu_k + s + 1);
  const bool ok = w.q0 >= 0 && w.q0 <= q1 && q1 <= a.num_q && w.k0 >= 0 && w.k0 <= k1 && k1 <= a.num_k;
  if (ok) {
    w.nq = q1 - w.q0;
    w.nk = k1 - w.k0;
  } else {
    w.q0 = min(max(w.q0, 0), a.num_q);
    w.k0 = min(max(w.k0, 0), a.num_k);
    w.nq = KEYS ? 0 : max(min(q1, a.num_q) - w.q0, 0);
    w.nk = KEYS ? max(min(k1, a.num_k) - w.k0, 0) : 0;
  }
  return w;
}

cudaError_t launch_prompt(const PromptArgs& a, bool half, cudaStream_t stream);
cudaError_t launch_prompt_bwd(const PromptArgs& a, bool half, cudaStream_t stream);

}  // namespace csa
