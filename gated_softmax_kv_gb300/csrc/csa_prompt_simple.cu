// Causal attention over packed sequences, the plain way: a warp a row.
//
// Forward and dq: a warp a (token, head), one key after the other, the running
// maximum and sum of a softmax. dk and dv: a warp a (key, key head), one query row
// after the other. Bound by instructions: five shuffles a pair.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "csa_device.cuh"
#include "csa_internal.h"
#include "csa_prompt_internal.h"
#include "csa_turn.cuh"

namespace csa {

namespace {

constexpr int C = 4;  // columns a lane: 32 * C >= 128

template <typename E>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int d, int lane, float (&v)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = lane + 32 * c < d ? Elem<E>::load(static_cast<const E*>(base) + at + lane + 32 * c) : 0.0f;
}
template <typename E>
__device__ __forceinline__ void store_row(void* base, int64_t at, int d, int lane, const float (&v)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (lane + 32 * c < d) Elem<E>::store(static_cast<E*>(base) + at + lane + 32 * c, v[c]);
}
__device__ __forceinline__ float dot(const float (&a)[C], const float (&b)[C]) {
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) s = fmaf(a[c], b[c], s);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// The last s with cu[s] <= t, or -1 for a row of no sequence.
__device__ __forceinline__ int seq_of(const int32_t* cu, int nseq, int t) {
  if (t < __ldg(cu) || t >= __ldg(cu + nseq)) return -1;
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <typename E, bool BWD>
__global__ void __launch_bounds__(128) rows_kernel(const PromptArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.num_q * a.heads;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * 4) {
    const int t = (int)(r / a.heads), h = (int)(r - (int64_t)t * a.heads), kvh = h / a.group;
    const int s = seq_of(a.cu_q, a.nseq, t);
    float o[C] = {};
    const Span w = s >= 0 ? span_of(a, s) : Span{0, 0, 0, 0};
    if (s < 0 || w.nq == 0) {
      if (BWD) {
        store_row<E>(a.dq, r * a.d, a.d, lane, o);
      } else {
        if (a.fill & CSA_FILL_OUT) store_row<E>(a.out, r * a.d, a.d, lane, o);
        if ((a.fill & CSA_FILL_OUT) && a.rest) store_row<E>(a.rest, r * a.d, a.d, lane, o);
        if ((a.fill & CSA_FILL_LSE) && lane == 0) a.lse[r] = -INFINITY;
      }
      continue;
    }
    const int last = w.nk - w.nq + (t - w.q0);
    const int first = a.window ? max(0, last + 1 - a.window) : 0;
    float q[C], k[C], v[C];
    load_row<E>(a.q, t * a.qt + h * a.qh, a.d, lane, q);
    if constexpr (!BWD) {
      float m = -INFINITY, l = 0.0f;
      for (int j = first; j <= last; ++j) {
        load_row<E>(a.k, (int64_t)(w.k0 + j) * a.kt + kvh * a.kh, a.d, lane, k);
        load_row<E>(a.v, (int64_t)(w.k0 + j) * a.vt + kvh * a.vh, a.d, lane, v);
        const float z = dot(q, k) * a.scale;
        const float top = fmaxf(m, z), safe = top == -INFINITY ? 0.0f : top;
        const float f = expf(m - safe), p = expf(z - safe);
        l = l * f + p;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = fmaf(p, v[c], o[c] * f);
        m = top;
      }
      float low[C];
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = l > 0.0f || l != l ? o[c] / l : 0.0f;
      store_row<E>(a.out, r * a.d, a.d, lane, o);
      if (a.rest) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          E x;
          Elem<E>::store(&x, o[c]);
          low[c] = o[c] - Elem<E>::load(&x);
        }
        store_row<E>(a.rest, r * a.d, a.d, lane, low);
      }
      if (lane == 0) a.lse[r] = l > 0.0f || l != l ? m + logf(l) : -INFINITY;
    } else {
      float g[C], x[C], y[C] = {};
      load_row<E>(a.g, t * a.gt + h * a.gh, a.d, lane, g);
      load_row<E>(a.out, r * a.d, a.d, lane, x);
      if (a.rest) load_row<E>(a.rest, r * a.d, a.d, lane, y);
      float delta = dot(g, x) + dot(g, y);
      const float dl = a.grad_lse ? a.grad_lse[r] : 0.0f, lse = a.lse[r];
      for (int j = first; j <= last; ++j) {
        load_row<E>(a.k, (int64_t)(w.k0 + j) * a.kt + kvh * a.kh, a.d, lane, k);
        load_row<E>(a.v, (int64_t)(w.k0 + j) * a.vt + kvh * a.vh, a.d, lane, v);
        const float p = lse == -INFINITY ? 0.0f : expf(dot(q, k) * a.scale - lse);
        const float ds = p * ((first == last ? 0.0f : dot(g, v) - delta) + dl);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = fmaf(ds, k[c], o[c]);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= a.scale;
      store_row<E>(a.dq, r * a.d, a.d, lane, o);
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(128) keys_kernel(const PromptArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.num_k * a.kv;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * 4) {
    const int t = (int)(r / a.kv), kvh = (int)(r - (int64_t)t * a.kv);
    const int s = seq_of(a.cu_k, a.nseq, t);
    float dk[C] = {}, dv[C] = {}, k[C], v[C], q[C], g[C], x[C], y[C] = {};
    if (s >= 0) {
      const Span w = span_of(a, s);
      const int j = t - w.k0, off = w.nk - w.nq;
      load_row<E>(a.k, t * a.kt + kvh * a.kh, a.d, lane, k);
      load_row<E>(a.v, t * a.vt + kvh * a.vh, a.d, lane, v);
      const int64_t i1 = a.window ? min((int64_t)w.nq, (int64_t)j - off + a.window) : w.nq;
      for (int64_t i = max(0, j - off); i < i1; ++i)
        for (int h = kvh * a.group; h < (kvh + 1) * a.group; ++h) {
          const int64_t qr = (w.q0 + i) * a.heads + h;
          load_row<E>(a.q, (w.q0 + i) * a.qt + h * a.qh, a.d, lane, q);
          load_row<E>(a.g, (w.q0 + i) * a.gt + h * a.gh, a.d, lane, g);
          load_row<E>(a.out, qr * a.d, a.d, lane, x);
          if (a.rest) load_row<E>(a.rest, qr * a.d, a.d, lane, y);
          const int last = off + (int)i, first = a.window ? max(0, last + 1 - a.window) : 0;
          const float lse = a.lse[qr], dl = a.grad_lse ? a.grad_lse[qr] : 0.0f;
          const float p = lse == -INFINITY ? 0.0f : expf(dot(q, k) * a.scale - lse);
          const float ds = p * ((first == last ? 0.0f : dot(g, v) - dot(g, x) - dot(g, y)) + dl);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            dk[c] = fmaf(ds * a.scale, q[c], dk[c]);
            dv[c] = fmaf(p, g[c], dv[c]);
          }
        }
    }
    store_row<E>(a.dk, r * a.d, a.d, lane, dk);
    store_row<E>(a.dv, r * a.d, a.d, lane, dv);
  }
}

}  // namespace

cudaError_t launch_prompt_bwd(const PromptArgs& a, bool half, cudaStream_t stream) {
  const dim3 grid(152 * 16), block(128);
  cudaError_t e = half ? launch_dependent(rows_kernel<__half, true>, grid, block, 0, stream, a)
                       : launch_dependent(rows_kernel<Bf16, true>, grid, block, 0, stream, a);
  if (e != cudaSuccess) return e;
  return half ? launch_dependent(keys_kernel<__half>, grid, block, 0, stream, a)
              : launch_dependent(keys_kernel<Bf16>, grid, block, 0, stream, a);
}

}  // namespace csa
