// Causal attention over packed sequences (declared in include/csa_prompt.h): the
// calls' checks. Kernels: csa_prompt_fwd.cu, csa_prompt_bwd.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "csa_cache_internal.h"
#include "csa_internal.h"
#include "csa_prompt_internal.h"
#include "csa_prompt_tile.cuh"

namespace csa {

// The encoder is a driver call, looked up once through the runtime.
cudaError_t rows_map(CUtensorMap* map, const void* base, bool half, int32_t d, int32_t heads, int64_t tokens, int64_t ts,
                     int64_t hs, int32_t heads_box, int32_t tokens_box) {
  using Encode = decltype(&cuTensorMapEncodeTiled);  // its type alone: nothing links against the driver
  static std::atomic<void*> known{nullptr};
  void* fn = known.load();
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    known.store(fn);
  }
  const Encode encode = reinterpret_cast<Encode>(fn);
  // a tensor without rows is never loaded from, but has a map; strides of single
  // elements are never stepped
  static const uint4 none = {};
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)(tokens > 0 ? tokens : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)(hs > 0 ? hs : 8) * 2, (cuuint64_t)(ts > 0 ? ts : 8) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)tokens_box}, steps[3] = {1, 1, 1};
  const CUresult r = encode(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                            const_cast<void*>(tokens > 0 ? base : &none), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Strides of [tokens, heads, head_dim] rows in elements of 2 bytes: multiples of 16
// bytes, above 0 and below 2^40 bytes where they are stepped.
csa_status_t check_strides(int64_t tokens, int64_t heads, int64_t ts, int64_t hs) {
  const int64_t most = ((int64_t)1 << 39) - 8;
  if ((tokens > 1 && (ts <= 0 || ts > most)) || (heads > 1 && (hs <= 0 || hs > most))) return CSA_ERR_RANGE;
  if ((tokens > 1 && ts % 8 != 0) || (heads > 1 && hs % 8 != 0)) return CSA_ERR_ALIGN;
  return CSA_OK;
}

csa_status_t check(const csa_prompt_t* p, PromptArgs& a) {
  if (!p) return CSA_ERR_NULL;
  if (p->dtype != CSA_BF16 && p->dtype != CSA_FP16) return CSA_ERR_UNSUPPORTED;
  if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8 != 0) return CSA_ERR_UNSUPPORTED;
  if (p->kv_heads < 1 || p->kv_heads > 65535 || p->heads < 1 || p->heads % p->kv_heads != 0 || p->heads / p->kv_heads > 128)
    return CSA_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)1 << 31;
  if (p->num_q < 0 || p->num_k < 0 || p->num_seqs < 1 || p->num_seqs > kMaxSeqs || p->window < 0) return CSA_ERR_RANGE;
  // tiles of rows are counted from token 0 in 31 bits
  if (p->num_q > lim - 4096 || p->num_k > lim - 4096 || p->num_q * p->heads >= lim || p->num_k * p->kv_heads >= lim)
    return CSA_ERR_RANGE;
  // tiles of both kernels, a grid each
  const int64_t tiles = (p->num_q > p->num_k ? p->num_q : p->num_k) + p->num_seqs;
  if (tiles * p->kv_heads >= lim) return CSA_ERR_RANGE;
  if (!(p->sm_scale > 0.0f) || !isfinite(p->sm_scale)) return CSA_ERR_RANGE;
  csa_status_t st = check_strides(p->num_q, p->heads, p->q_token_stride, p->q_head_stride);
  if (st == CSA_OK) st = check_strides(p->num_k, p->kv_heads, p->k_token_stride, p->k_head_stride);
  if (st == CSA_OK) st = check_strides(p->num_k, p->kv_heads, p->v_token_stride, p->v_head_stride);
  if (st != CSA_OK) return st;
  if (!p->cu_q || (p->num_q > 0 && !p->q) || (p->num_k > 0 && (!p->k || !p->v))) return CSA_ERR_NULL;
  if (!p->cu_k && p->num_q != p->num_k) return CSA_ERR_RANGE;
  if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || misaligned4(p->cu_q) || misaligned4(p->cu_k))
    return CSA_ERR_ALIGN;
  a = {};
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.cu_q = p->cu_q;
  a.cu_k = p->cu_k ? p->cu_k : p->cu_q;
  // the stride of a single element is never stepped
  a.qt = p->num_q > 1 ? p->q_token_stride : 0;
  a.qh = p->heads > 1 ? p->q_head_stride : 0;
  a.kt = p->num_k > 1 ? p->k_token_stride : 0;
  a.kh = p->kv_heads > 1 ? p->k_head_stride : 0;
  a.vt = p->num_k > 1 ? p->v_token_stride : 0;
  a.vh = p->kv_heads > 1 ? p->v_head_stride : 0;
  a.num_q = (int32_t)p->num_q;
  a.num_k = (int32_t)p->num_k;
  a.nseq = p->num_seqs;
  a.heads = p->heads;
  a.kv = p->kv_heads;
  a.group = p->heads / p->kv_heads;
  a.d = p->head_dim;
  a.window = p->window;
  a.scale = p->sm_scale;
  a.polls = csa_prompt_polls;
  return CSA_OK;
}

}  // namespace

}  // namespace csa

extern "C" int32_t csa_prompt_polls = csa::kPolls;

extern "C" csa_status_t csa_prompt_attend(const csa_prompt_t* p, void* out, void* rest, float* lse, int32_t fill,
                                          cudaStream_t stream) {
  csa::PromptArgs a;
  const csa_status_t st = csa::check(p, a);
  if (st != CSA_OK) return st;
  if (fill & ~(CSA_FILL_OUT | CSA_FILL_LSE)) return CSA_ERR_UNSUPPORTED;
  if (p->num_q > 0 && (!out || !lse)) return CSA_ERR_NULL;
  if (!csa::aligned16(out) || !csa::aligned16(rest) || csa::misaligned4(lse)) return CSA_ERR_ALIGN;
  if (p->num_q == 0) return CSA_OK;
  a.out = out;
  a.rest = rest;
  a.lse = lse;
  a.fill = fill;
  const cudaError_t e = csa::launch_prompt(a, p->dtype == CSA_FP16, stream);
  return e == cudaSuccess ? CSA_OK : csa::record_cuda_error(e);
}

extern "C" csa_status_t csa_prompt_attend_bwd(const csa_prompt_t* p, const void* out, const void* rest, const float* lse,
                                              const void* grad, int64_t grad_token_stride, int64_t grad_head_stride,
                                              const float* grad_lse, void* dq, void* dk, void* dv, cudaStream_t stream) {
  csa::PromptArgs a;
  csa_status_t st = csa::check(p, a);
  if (st == CSA_OK) st = csa::check_strides(p->num_q, p->heads, grad_token_stride, grad_head_stride);
  if (st != CSA_OK) return st;
  if ((p->num_q > 0 && (!out || !lse || !grad || !dq)) || (p->num_k > 0 && (!dk || !dv))) return CSA_ERR_NULL;
  if (!csa::aligned16(out) || !csa::aligned16(rest) || !csa::aligned16(grad) || !csa::aligned16(dq) || !csa::aligned16(dk) ||
      !csa::aligned16(dv) || csa::misaligned4(lse) || csa::misaligned4(grad_lse))
    return CSA_ERR_ALIGN;
  a.out = const_cast<void*>(out);
  a.rest = const_cast<void*>(rest);
  a.lse = const_cast<float*>(lse);
  a.g = grad;
  a.gt = p->num_q > 1 ? grad_token_stride : 0;
  a.gh = p->heads > 1 ? grad_head_stride : 0;
  a.grad_lse = grad_lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  cudaError_t e = cudaSuccess;
  if (p->num_q == 0) {  // no query: nothing reaches the keys
    const size_t bytes = (size_t)p->num_k * p->kv_heads * p->head_dim * 2;
    if (bytes > 0) e = cudaMemsetAsync(dk, 0, bytes, stream);
    if (bytes > 0 && e == cudaSuccess) e = cudaMemsetAsync(dv, 0, bytes, stream);
  } else {
    e = csa::launch_prompt_bwd(a, p->dtype == CSA_FP16, stream);
  }
  return e == cudaSuccess ? CSA_OK : csa::record_cuda_error(e);
}
