// csa_cache_attend (declared in include/csa_cache.h): argument checks and the
// choice of the kernel.
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache_attend.h"

extern "C" csa_status_t csa_cache_attend(const csa_cache_t* cache, const void* q, int32_t dtype,
                                         int64_t num_tokens, int32_t num_q_heads,
                                         int64_t q_token_stride, int64_t q_head_stride,
                                         int32_t kv_heads, int32_t shared, float sm_scale,
                                         const int32_t* page_table, int32_t num_seqs,
                                         int32_t max_pages, const int32_t* seq_lens,
                                         const int32_t* cu_q, const int32_t* visible, void* out,
                                         float* lse, cudaStream_t stream) {
  const csa_status_t st = csa::check_cache(cache);
  if (st != CSA_OK) return st;
  if (dtype != CSA_BF16 && dtype != CSA_FP16) return CSA_ERR_UNSUPPORTED;
  if (kv_heads < 1 || num_q_heads < 1 || num_q_heads > 65536 || num_q_heads % kv_heads != 0 ||
      (int64_t)kv_heads * (shared ? 1 : 2) > cache->num_heads)
    return CSA_ERR_UNSUPPORTED;
  if (num_seqs < 1 || num_seqs > csa::kMaxSeqs || max_pages < 1 || max_pages > csa::kMaxPages || num_tokens < 0 ||
      q_token_stride < 0 || q_head_stride < 0)
    return CSA_ERR_RANGE;
  if (num_tokens >= ((int64_t)1 << 31) || num_tokens * num_q_heads >= ((int64_t)1 << 31))
    return CSA_ERR_RANGE;
  const int64_t most = (int64_t)1 << 56;
  if (q_token_stride > most / (num_tokens + 1) || q_head_stride > most / (num_q_heads + 1))
    return CSA_ERR_RANGE;
  if (!page_table || !seq_lens || !cu_q || (num_tokens > 0 && (!q || !out))) return CSA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(q) % 16 != 0 || reinterpret_cast<uintptr_t>(out) % 16 != 0 ||
      q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || csa::misaligned4(page_table) ||
      csa::misaligned4(seq_lens) || csa::misaligned4(cu_q) || csa::misaligned4(visible) ||
      csa::misaligned4(lse))
    return CSA_ERR_ALIGN;
  if (num_tokens == 0) return CSA_OK;
  csa::AttendArgs a;
  a.c = csa::view_of(cache);
  a.q = static_cast<const uint16_t*>(q);
  a.tokens = num_tokens;
  a.qt = q_token_stride;
  a.qh = q_head_stride;
  a.heads = num_q_heads;
  a.kv = kv_heads;
  a.group = num_q_heads / kv_heads;
  a.v_first = shared ? 0 : kv_heads;
  a.scale = sm_scale * 1.4426950408889634f;
  a.table = page_table;
  a.lens = seq_lens;
  a.cu = cu_q;
  a.visible = visible;
  a.nseq = num_seqs;
  a.max_pages = max_pages;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.ws = nullptr;
  // By the query rows of a sequence and cache head, on average over the sequences.
  // The rows kernel passes over the keys once for 16 rows, the wide one for 64.
  // Measured (32 sequences of 4096 rows, as a graph, rows against wide kernel):
  // shared rows of 512 columns, 16 rows 34 us / 62, 32 rows 56 / 62, 64 rows
  // 102 / 64; two heads of 128 columns, 30 / 49, 46 / 49, 76 / 49; of 64 columns,
  // which fill half of the wide kernel's panels, 26 / 47, 38 / 49, 62 / 48.
  const int64_t most_rows = cache->head_dim == 64 ? 48 : 32;
  const bool wide = num_tokens * a.group > most_rows * num_seqs;
  const cudaError_t e = wide ? csa::launch_attend_wide(a, dtype == CSA_FP16, shared != 0, stream)
                             : csa::launch_attend_rows(a, dtype == CSA_FP16, shared != 0, stream);
  return e == cudaSuccess ? CSA_OK : csa::record_cuda_error(e);
}
