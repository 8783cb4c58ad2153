// csa_cache_attend (declared in include/csa_cache.h): attention over the
// paged 8-bit cache.
//
// The simplest form: one warp per (query token, head) walks the rows it sees
// with a running maximum and sum, lanes split the columns.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache_internal.h"
#include "csa_device.cuh"
#include "csa_e4m3.cuh"

namespace csa {

namespace {

struct AttendArgs {
  CacheView c;
  const uint16_t* q;
  int64_t tokens, qt, qh;
  int32_t heads, kv, group;
  int32_t v_first;  // cache head of the first value head
  float scale;      // sm_scale * log2 e
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  const int32_t* visible;
  int32_t nseq, max_pages;
  uint16_t* out;
  float* lse;
};

__device__ __forceinline__ int seq_of(const int32_t* cu, int nseq, int64_t t) {
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int D, bool HALF>
__global__ void __launch_bounds__(256) attend_simple_kernel(const AttendArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int N = D / 32;  // columns a lane
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = unit / a.heads;
  const int h = (int)(unit - t * a.heads);
  if (t >= a.tokens || t >= __ldg(a.cu + a.nseq) || t < __ldg(a.cu)) return;
  const int s = seq_of(a.cu, a.nseq, t);
  int64_t n = __ldg(a.lens + s);
  if (a.visible) n = min(n, (int64_t)__ldg(a.visible + t));
  n = min(n, (int64_t)a.max_pages << a.c.page_bits);
  const int kh = h / a.group, vh = a.v_first + kh;
  float q[N], o[N], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < N; ++i) {
    const uint16_t w = a.q[t * a.qt + h * a.qh + lane * N + i];
    q[i] = HALF ? __half2float(__ushort_as_half(w)) : __uint_as_float((uint32_t)w << 16);
    o[i] = 0.0f;
  }
  const int pb = a.c.page_bits, bb = a.c.block_bits;
  for (int64_t j = 0; j < n; ++j) {
    const int32_t page = __ldg(a.table + (int64_t)s * a.max_pages + (j >> pb));
    if (page < 0 || page >= a.c.num_pages) continue;
    const int slot = (int)(j & ((1 << pb) - 1));
    const int64_t kc = (int64_t)page * a.c.heads + kh, vc = (int64_t)page * a.c.heads + vh;
    const uint8_t* kp = a.c.data + ((kc << pb) + slot) * D + lane * N;
    const uint8_t* vp = a.c.data + ((vc << pb) + slot) * D + lane * N;
    const float ks = a.c.scales[(kc << (pb - bb)) + (slot >> bb)];
    const float vs = a.c.scales[(vc << (pb - bb)) + (slot >> bb)];
    float z = 0.0f, v[N];
    for (int i = 0; i < N; i += 2) {
      const uint32_t kk = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kp + i));
      const uint32_t vv = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vp + i));
      const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kk));
      const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&vv));
      z = fmaf(q[i], kf.x, fmaf(q[i + 1], kf.y, z));
      v[i] = vf.x;
      v[i + 1] = vf.y;
    }
    for (int x = 16; x; x >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, x);
    z *= ks * a.scale;
    const float m2 = fmaxf(m, z);
    const float ref = m2 == -INFINITY ? 0.0f : m2;
    const float f = exp2f(m - ref), p = exp2f(z - ref);
    l = l * f + p;
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + (p * vs) * v[i];
    m = m2;
  }
  const bool none = l == 0.0f;
  for (int i = 0; i < N; ++i) {
    const float r = none ? 0.0f : o[i] / l;
    a.out[(t * a.heads + h) * D + lane * N + i] =
        HALF ? __half_as_ushort(__float2half_rn(r)) : (uint16_t)(pack_bf16x2(r, 0.0f) & 0xFFFFu);
  }
  if (a.lse && lane == 0)
    a.lse[t * a.heads + h] = none ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

template <int D>
cudaError_t launch_attend(const AttendArgs& a, int dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.tokens * a.heads + 7) / 8));
  return dtype == CSA_FP16
             ? launch_dependent(attend_simple_kernel<D, true>, grid, dim3(256), 0, stream, a)
             : launch_dependent(attend_simple_kernel<D, false>, grid, dim3(256), 0, stream, a);
}

}  // namespace

}  // namespace csa

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
  if (num_seqs < 1 || num_seqs > csa::kMaxSeqs || max_pages < 1 || num_tokens < 0 ||
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
  cudaError_t e;
  switch (cache->head_dim) {
    case 64: e = csa::launch_attend<64>(a, dtype, stream); break;
    case 128: e = csa::launch_attend<128>(a, dtype, stream); break;
    case 256: e = csa::launch_attend<256>(a, dtype, stream); break;
    default: e = csa::launch_attend<512>(a, dtype, stream); break;
  }
  return e == cudaSuccess ? CSA_OK : csa::record_cuda_error(e);
}
