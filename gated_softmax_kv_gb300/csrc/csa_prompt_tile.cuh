// Shared by the tcgen05 kernels of causal attention over packed sequences: tiles of
// query rows, what they see, and cleaning of operands. Not installed.
//
// A tile is 128 rows of the matrix instructions: `tp` tokens by the `group` query
// heads of a key head (row = token * group + head), so that heads that share keys
// share a tile whatever their number, and the keys are read once for all of them.
// tp = 128 / group; rows at or behind tp * group are not used.
//
// Which tile is whose: slot(s) = floor(cu[s] / B) + s is the first slot of sequence
// s for stretches of B tokens, since ceil(n / B) <= floor((c + n) / B) - floor(c / B)
// + 1. So a CTA finds its sequence by searching cu, with no prefix sums and at most
// one slot a sequence that has no work.
#pragma once

#include <cuda_fp16.h>

#include "csa_device.cuh"
#include "csa_prompt_internal.h"
#include "csa_tc.cuh"

namespace csa {

__device__ __forceinline__ int64_t first_slot(const int32_t* cu, int s, int b) {
  return (int64_t)(max(__ldg(cu + s), 0) / b) + s;
}

// The last s in [0, nseq) whose first slot is at or before `slot`, by a warp, 32 at
// a time.
__device__ __forceinline__ int seq_of_slot(const int32_t* cu, int nseq, int b, int64_t slot, int lane) {
  int lo = 0, span = nseq;
  while (span > 1) {
    const int step = (span + 31) / 32, at = lo + lane * step;
    const bool before = lane * step < span && first_slot(cu, at, b) <= slot;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, before);
    const int k = who ? 31 - __clz(who) : 0;
    span = min(step, span - k * step);
    lo += k * step;
  }
  return lo;
}

// Rows of no sequence: [0, cu[0]) and [cu[nseq], n), a thread's share (every `step`-th
// from `from` on) of `words` 16-byte vectors of zeros a row.
__device__ __forceinline__ void fill_rest(const int32_t* cu, int nseq, int32_t n, int64_t words, uint4* to, int64_t from,
                                          int64_t step) {
  const int64_t a = min(max(__ldg(cu), 0), n), b = max((int64_t)min(max(__ldg(cu + nseq), 0), n), a);
#pragma unroll 1
  for (int64_t i = from; i < (a + n - b) * words; i += step) {
    const int64_t row = i / words;
    to[row < a ? i : i + (b - a) * words] = make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void fill_rest(const int32_t* cu, int nseq, int32_t n, int32_t heads, float v, float* to,
                                          int64_t from, int64_t step) {
  const int64_t a = min(max(__ldg(cu), 0), n), b = max((int64_t)min(max(__ldg(cu + nseq), 0), n), a);
#pragma unroll 1
  for (int64_t i = from; i < (a + n - b) * heads; i += step)
    to[i / heads < a ? i : i + (b - a) * heads] = v;
}

// Half a word pair whose exponent is all ones: infinity or NaN.
template <bool HALF>
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {
  constexpr uint32_t E = HALF ? 0x7C00u : 0x7F80u;
  uint32_t keep = 0;
  if ((w & E) != E) keep |= 0xFFFFu;
  if ((w & (E << 16)) != (E << 16)) keep |= 0xFFFF0000u;
  return keep;
}
template <bool HALF>
__device__ __forceinline__ bool all_finite(uint4 v) {
  return (finite_mask<HALF>(v.x) & finite_mask<HALF>(v.y) & finite_mask<HALF>(v.z) & finite_mask<HALF>(v.w)) ==
         0xFFFFFFFFu;
}

// Zeros for infinities and NaN in an operand's `bytes` of shared memory, by `threads`
// threads of which this is one; *found is set where there were any. A weight of 0 keeps
// a finite value out of a sum, but not these.
template <bool HALF>
__device__ __noinline__ void clean_operand(uint8_t* at, int bytes, int thread, int threads, volatile int32_t* found) {
  bool any = false;
#pragma unroll 1
  for (int i = thread * 16; i < bytes; i += threads * 16) {
    uint4* p = reinterpret_cast<uint4*>(at + i);
    const uint4 v = *p;
    if (!all_finite<HALF>(v)) {
      *found = 1;
      __threadfence_block();
      *p = make_uint4(v.x & finite_mask<HALF>(v.x), v.y & finite_mask<HALF>(v.y), v.z & finite_mask<HALF>(v.z),
                      v.w & finite_mask<HALF>(v.w));
      any = true;
    }
  }
  if (__any_sync(0xFFFFFFFFu, any)) fence_async();
}

template <bool HALF>
__device__ __forceinline__ float value16(uint16_t b) {
  return HALF ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (HALF) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return pack_bf16x2(lo, hi);
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 32 bytes, a sector, at once.
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A tensor map of [tokens, heads, d] rows: boxes of 64 columns, `heads_box` heads and
// `tokens_box` tokens. (csa_prompt.cu)
cudaError_t rows_map(CUtensorMap* map, const void* base, bool half, int32_t d, int32_t heads, int64_t tokens, int64_t ts,
                     int64_t hs, int32_t heads_box, int32_t tokens_box);

}  // namespace csa
