// Shared by the cache's translation units (csa_cache_append.cu,
// csa_cache_attend.cu, csa_cache_pages.cu). Not installed, not part of the
// ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache.h"
#include "csa_internal.h"

namespace csa {

constexpr int32_t kMaxSeqs = 262144;
constexpr int32_t kMaxPages = 1 << 27;  // of a table row: 2^31 rows of the smallest pages

// Envelope, alignment and pointers of a cache description.
inline csa_status_t check_cache(const csa_cache_t* c) {
  if (!c) return CSA_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256 && c->head_dim != 512)
    return CSA_ERR_UNSUPPORTED;
  const int32_t p = c->page_size, b = c->block;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) return CSA_ERR_UNSUPPORTED;
  if (b < 1 || b > p || (b & (b - 1)) != 0) return CSA_ERR_UNSUPPORTED;
  if (c->num_heads < 1 || c->num_heads > 1024) return CSA_ERR_UNSUPPORTED;
  if (c->num_pages < 1 || c->num_pages > (1 << 24)) return CSA_ERR_RANGE;
  if (!c->data || !c->scales) return CSA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(c->data) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(c->scales) % 4 != 0)
    return CSA_ERR_ALIGN;
  return CSA_OK;
}

inline bool misaligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

inline int log2_of(int32_t v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

// Stream-ordered device workspace from the library's pool (csa_api.cu).
cudaError_t workspace_take(void** ptr, size_t bytes, cudaStream_t stream);
cudaError_t workspace_give(void* ptr, cudaStream_t stream);

// The cache as kernels take it.
struct CacheView {
  uint8_t* data;
  float* scales;
  int32_t num_pages;
  int32_t heads;
  int32_t page_bits;   // log2 page_size
  int32_t block_bits;  // log2 block
  int32_t d;
};

inline CacheView view_of(const csa_cache_t* c) {
  CacheView v;
  v.data = static_cast<uint8_t*>(c->data);
  v.scales = c->scales;
  v.num_pages = c->num_pages;
  v.heads = c->num_heads;
  v.page_bits = log2_of(c->page_size);
  v.block_bits = log2_of(c->block);
  v.d = c->head_dim;
  return v;
}

}  // namespace csa
