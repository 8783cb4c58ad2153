// Shared by the attention's translation units (csa_cache_attend.cu and the
// kernels). Not installed, not part of the ABI.
#pragma once

#include "csa_cache_internal.h"

namespace csa {

struct AttendArgs {
  CacheView c;
  const uint16_t* q;
  int64_t tokens, qt, qh;   // q strides in elements
  int32_t heads, kv, group; // group: query heads of a cache head
  int32_t v_first;          // cache head of the first value head
  float scale;              // sm_scale * log2 e
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  const int32_t* visible;
  int32_t nseq, max_pages;
  uint16_t* out;
  float* lse;
  float* ws;                // partial results of split items
};

// Tiles of up to 16 query rows on mma.sync (csa_cache_attend_rows.cu).
cudaError_t launch_attend_rows(const AttendArgs& a, bool half, bool shared, cudaStream_t stream);
// Tiles of 64 query rows on tcgen05 (csa_cache_attend_wide.cu).
cudaError_t launch_attend_wide(const AttendArgs& a, bool half, bool shared, cudaStream_t stream);

}  // namespace csa
