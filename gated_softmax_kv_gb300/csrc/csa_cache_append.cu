// csa_cache_append (declared in include/csa_cache.h): quantises new rows into
// the pages of the 8-bit cache.
//
// One group of threads owns one (sequence, block of rows, head): it takes the
// maximum of |x| over the new rows of the block, settles the block's scale,
// requantises the rows that were there if the scale grew, and writes the new
// ones, so nothing is shared between groups and no order matters. The second
// pass finds the rows in L1 (a task is 64 KB at most for 64 rows of 512 bf16
// columns); keeping them in registers instead left two CTAs an SM and took 33 us
// for 79144 such rows, this 27 (4.5 TB/s, 66% of the copy rate). Bound by memory:
// 2 bytes read and 1 written a value for 16-bit rows; what keeps it from the rate
// is that a task's values wait for its maximum.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache_internal.h"
#include "csa_device.cuh"
#include "csa_e4m3.cuh"

namespace csa {

namespace {

struct AppendArgs {
  CacheView c;
  const void* rows;
  int64_t num_rows, row_stride, head_stride;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int32_t nseq, max_pages;
  int64_t tasks;
};

template <int DTYPE>
struct Row16;  // 16 bytes of the rows' type
template <>
struct Row16<CSA_BF16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float at(const uint4& w, int i) {
    const uint32_t u = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
    return bf16_at(u, i & 1);
  }
};
template <>
struct Row16<CSA_FP16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float at(const uint4& w, int i) {
    const uint32_t u = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
    return __half2float(__ushort_as_half((unsigned short)(i & 1 ? u >> 16 : u & 0xFFFFu)));
  }
};
template <>
struct Row16<CSA_FP32> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float at(const uint4& w, int i) {
    return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
  }
};

// Magnitudes are compared as integers: without the sign, the bits of each type
// grow with the value, infinities and NaN above every finite one. 16-bit types
// go two to an instruction.
template <int DTYPE>
struct Magnitude {
  static constexpr uint32_t INF = DTYPE == CSA_BF16 ? 0x7F80u : DTYPE == CSA_FP16 ? 0x7C00u : 0x7F800000u;
  static constexpr bool PACKED = DTYPE != CSA_FP32;
  // the larger of m and the vector's magnitudes (a pair of maxima for 16-bit types)
  static __device__ __forceinline__ uint32_t max_of(uint32_t m, const uint4& w) {
    if constexpr (PACKED) {
      m = __vmaxu2(m, __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu));
      return __vmaxu2(m, __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    } else {
      m = max(m, max(w.x & 0x7FFFFFFFu, w.y & 0x7FFFFFFFu));
      return max(m, max(w.z & 0x7FFFFFFFu, w.w & 0x7FFFFFFFu));
    }
  }
  // the same over the finite ones
  static __device__ __forceinline__ uint32_t finite_max_of(uint32_t m, const uint4& w) {
#pragma unroll
    for (int i = 0; i < Row16<DTYPE>::N; ++i) {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      const uint32_t b = PACKED ? (u[i / 2] >> (16 * (i & 1))) & 0x7FFFu : u[i] & 0x7FFFFFFFu;
      if (b < INF) m = max(m, b);
    }
    return m;
  }
  static __device__ __forceinline__ float value(uint32_t bits) {
    return DTYPE == CSA_BF16   ? __uint_as_float(bits << 16)
           : DTYPE == CSA_FP16 ? __half2float(__ushort_as_half((unsigned short)bits))
                               : __uint_as_float(bits);
  }
};

// One vector times the inverse scale, as e4m3. The product is exact (a power
// of two) wherever it matters: below 2^-126 it rounds to an e4m3 zero anyway.
template <int DTYPE, bool FINITE>
__device__ __forceinline__ void store_quantised(uint8_t* p, const uint4& w, float inv) {
  constexpr int N = Row16<DTYPE>::N;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float x = Row16<DTYPE>::at(w, i);
    v[i] = FINITE || fabsf(x) < INFINITY ? x * inv : NAN;  // infinities have no e4m3 value
  }
  if constexpr (N == 8) {
    uint2 o;
    o.x = e4m3x4_of(v[0], v[1], v[2], v[3]);
    o.y = e4m3x4_of(v[4], v[5], v[6], v[7]);
    *reinterpret_cast<uint2*>(p) = o;
  } else {
    *reinterpret_cast<uint32_t*>(p) = e4m3x4_of(v[0], v[1], v[2], v[3]);
  }
}

// THREADS 256: a CTA owns a task; THREADS 32: each of a CTA's 8 warps does.
template <int DTYPE, int THREADS>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int N = Row16<DTYPE>::N;
  __shared__ uint32_t warp_max[8];
  const int lane = THREADS == 256 ? threadIdx.x : threadIdx.x & 31;
  const int64_t unit = THREADS == 256 ? (int64_t)blockIdx.x
                                      : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t task = unit / a.c.heads;
  const int head = (int)(unit - task * a.c.heads);
  if (task >= a.tasks) return;

  // Sequence s owns the tasks from cu[s] / block + 2 s on: n rows touch at
  // most n / block + 2 blocks.
  const int bb = a.c.block_bits, pb = a.c.page_bits;
  int lo = 0, hi = a.nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (((int64_t)__ldg(a.cu + mid) >> bb) + 2 * (int64_t)mid <= task)
      lo = mid;
    else
      hi = mid;
  }
  const int s = lo;
  const int64_t c0 = __ldg(a.cu + s), c1 = __ldg(a.cu + s + 1);
  const int64_t held = __ldg(a.lens + s);
  if (c0 < 0 || c1 > a.num_rows || c1 <= c0 || held < 0) return;
  const int64_t local = task - ((c0 >> bb) + 2 * (int64_t)s);
  const int64_t begin = ((held >> bb) + local) << bb;  // first row of the block
  const int64_t first = begin > held ? begin : held;
  const int64_t stop = held + (c1 - c0);
  const int64_t last = stop < begin + (1 << bb) ? stop : begin + (1 << bb);
  if (local < 0 || first >= last) return;
  const int64_t entry = begin >> pb;
  if (entry >= a.max_pages) return;
  const int32_t page = __ldg(a.table + (int64_t)s * a.max_pages + entry);
  if (page < 0 || page >= a.c.num_pages) return;

  const int slot0 = (int)(begin & ((1 << pb) - 1));
  const int64_t chunk = (int64_t)page * a.c.heads + head;
  uint8_t* data = a.c.data + ((chunk << pb) + slot0) * a.c.d;  // the block's first row
  float* scale = a.c.scales + (chunk << (pb - bb)) + (slot0 >> bb);
  const uint8_t* src = static_cast<const uint8_t*>(a.rows) +
                       ((c0 + first - held) * a.row_stride + head * a.head_stride) * (16 / N);
  const int64_t src_row = a.row_stride * (16 / N);
  const int per_row = a.c.d / N;  // a power of two
  const int row_bits = 31 - __clz(per_row);
  const int vecs = (int)(last - first) << row_bits;

  auto vec = [&](int v) {
    return reinterpret_cast<const uint4*>(src + (v >> row_bits) * src_row) + (v & (per_row - 1));
  };
  using Mag = Magnitude<DTYPE>;
  // the group's maximum of a thread's
  auto group_max = [&](uint32_t m) {
    if (Mag::PACKED) m = max(m >> 16, m & 0xFFFFu);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if constexpr (THREADS == 256) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) m = max(m, warp_max[w]);
    }
    return m;
  };
  const bool begun = first > begin;
  const float old = begun ? *scale : 0.0f;
  uint32_t top = 0;
  for (int v = lane; v < vecs; v += 4 * THREADS) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v + k * THREADS < vecs ? __ldg(vec(v + k * THREADS)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) top = Mag::max_of(top, x[k]);
  }
  top = group_max(top);  // for a CTA, also: every thread has read the old scale
  const bool finite = top < Mag::INF;
  if (!finite) {
    top = 0;
    for (int v = lane; v < vecs; v += THREADS) top = Mag::finite_max_of(top, __ldg(vec(v)));
    top = group_max(top);
  }
  __syncwarp();
  const float m = Mag::value(top);
  const float need = exp2i(scale_exp(m));
  const bool grew = !begun || need > old;
  const float now = grew ? need : old;
  if (grew && lane == 0) *scale = now;
  if (begun && grew) {
    const float f = old / now;
    const int words = ((int)(first - begin) * a.c.d) >> 2;
    uint32_t* w = reinterpret_cast<uint32_t*>(data);
    for (int i = lane; i < words; i += THREADS) {
      float v[4];
      e4m3x4_to_f32(w[i], v);
      w[i] = e4m3x4_of(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    }
  }
  const float inv = 1.0f / now;
  uint8_t* dst = data + (int64_t)(first - begin) * a.c.d;
  for (int v = lane; v < vecs; v += 4 * THREADS) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v + k * THREADS < vecs) x[k] = __ldg(vec(v + k * THREADS));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v + k * THREADS < vecs) {
        uint8_t* p = dst + (int64_t)(v + k * THREADS) * N;
        if (finite)
          store_quantised<DTYPE, true>(p, x[k], inv);
        else
          store_quantised<DTYPE, false>(p, x[k], inv);
      }
  }
}

template <int DTYPE>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  // A block of more than 8192 values keeps a CTA's threads busy; smaller ones would
  // leave most of them idle and take a warp. Measured (79144 bf16 rows, as a graph,
  // CTA against warp): 64 rows of 512 columns 24 us / 53, 32 of 512 25 / 31, 64 of
  // 256 13 / 17, 16 of 512 28 / 23, 64 of 128 9.1 / 9.8, 64 of 64 8.2 / 6.3, 16 of
  // 64 19.5 / 5.7.
  const int64_t units = a.tasks * a.c.heads;
  if (((int64_t)a.c.d << a.c.block_bits) > 8192)
    return launch_dependent(append_kernel<DTYPE, 256>, dim3((unsigned)units), dim3(256), 0, stream,
                            a);
  return launch_dependent(append_kernel<DTYPE, 32>, dim3((unsigned)((units + 7) / 8)), dim3(256), 0,
                          stream, a);
}

}  // namespace

}  // namespace csa

extern "C" csa_status_t csa_cache_append(const csa_cache_t* cache, const void* rows, int32_t dtype,
                                         int64_t num_rows, int64_t row_stride, int64_t head_stride,
                                         const int32_t* page_table, int32_t num_seqs,
                                         int32_t max_pages, const int32_t* seq_lens,
                                         const int32_t* cu_rows, cudaStream_t stream) {
  const csa_status_t st = csa::check_cache(cache);
  if (st != CSA_OK) return st;
  if (dtype != CSA_BF16 && dtype != CSA_FP16 && dtype != CSA_FP32) return CSA_ERR_UNSUPPORTED;
  if (num_seqs < 1 || num_seqs > csa::kMaxSeqs || max_pages < 1 || max_pages > csa::kMaxPages || num_rows < 0 ||
      num_rows >= ((int64_t)1 << 31) || row_stride < 0 || head_stride < 0)
    return CSA_ERR_RANGE;
  const int64_t most = (int64_t)1 << 56;
  if (row_stride > most / (num_rows + 1) || head_stride > most / (cache->num_heads + 1))
    return CSA_ERR_RANGE;
  if (!page_table || !seq_lens || !cu_rows || (num_rows > 0 && !rows)) return CSA_ERR_NULL;
  const int per = dtype == CSA_FP32 ? 4 : 8;
  if (reinterpret_cast<uintptr_t>(rows) % 16 != 0 || row_stride % per != 0 ||
      head_stride % per != 0 || csa::misaligned4(page_table) || csa::misaligned4(seq_lens) ||
      csa::misaligned4(cu_rows))
    return CSA_ERR_ALIGN;
  if (num_rows == 0) return CSA_OK;
  csa::AppendArgs a;
  a.c = csa::view_of(cache);
  a.rows = rows;
  a.num_rows = num_rows;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  a.table = page_table;
  a.lens = seq_lens;
  a.cu = cu_rows;
  a.nseq = num_seqs;
  a.max_pages = max_pages;
  a.tasks = (num_rows >> a.c.block_bits) + 2 * (int64_t)num_seqs;
  if (a.tasks * a.c.heads >= ((int64_t)1 << 31)) return CSA_ERR_RANGE;
  const cudaError_t e = dtype == CSA_BF16   ? csa::launch_append<CSA_BF16>(a, stream)
                        : dtype == CSA_FP16 ? csa::launch_append<CSA_FP16>(a, stream)
                                            : csa::launch_append<CSA_FP32>(a, stream);
  return e == cudaSuccess ? CSA_OK : csa::record_cuda_error(e);
}
