// What the attention's kernels share: the numbers that the numerics rest on
// (csa_cache_attend_rows.cu), the joining of partial results and the writing of
// finished rows.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "csa_cache_attend.h"
#include "csa_cache_plan.cuh"
#include "csa_device.cuh"
#include "csa_e4m3.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;     // of the joining kernel and of attend_rows_kernel
constexpr float kNone = -1e38f;   // reference before the first logit
constexpr float kSlackM = 60.0f;  // how far logits may pass m
constexpr float kSlackW = 8.0f;   // and z + log2 s pass m'
constexpr float kLift = 7.0f;     // weights carry 2^7

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lo_f16x2(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_f16x2(uint32_t w) {
  return e4m3x2_to_f16x2((uint16_t)(w >> 16));
}
// A query row as fp16, times a power of two that puts its largest finite value
// into [2^14, 2^15) (as far as 2^126 reaches). A lane holds V vectors of it.
// The magnitudes are compared as integers, two to an instruction: without the
// sign, the bits grow with the value, infinities and NaN above every finite one.
template <bool HALF, int V>
__device__ __forceinline__ uint32_t finite_max(const uint4 (&x)[V]) {
  constexpr uint32_t INF = HALF ? 0x7C00u : 0x7F80u;
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    m = __vmaxu2(m, __vmaxu2(x[k].x & 0x7FFF7FFFu, x[k].y & 0x7FFF7FFFu));
    m = __vmaxu2(m, __vmaxu2(x[k].z & 0x7FFF7FFFu, x[k].w & 0x7FFF7FFFu));
  }
  m = max(m >> 16, m & 0xFFFFu);
  if (__any_sync(0xFFFFFFFFu, m >= INF)) {
    m = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = (u[e >> 1] >> (16 * (e & 1))) & 0x7FFFu;
        if (b < INF) m = max(m, b);
      }
    }
  }
  return __reduce_max_sync(0xFFFFFFFFu, m);
}
// The power: the bits of finite_max to the exponent.
template <bool HALF>
__device__ __forceinline__ int query_lift(uint32_t amax) {
  if (amax == 0) return 0;
  const float v = HALF ? __half2float(__ushort_as_half((unsigned short)amax)) : __uint_as_float(amax << 16);
  return min(14 + 127 - (int)(__float_as_uint(v) >> 23), 126);
}
template <bool HALF>
__device__ __forceinline__ uint4 lifted(const uint4& x, float f) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 v;
    if (HALF)
      v = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
    else
      v = make_float2(bf16_lo(u[e]), bf16_hi(u[e]));
    r[e] = pack_f16x2(v.x * f, v.y * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// 0xFF in the bytes that hold a NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

struct RowStats {
  float m, mp, l;
};

// out = sum * 2^(m' - m - 7) / l, in one exponential.
__device__ __forceinline__ float out_factor(const RowStats& r) {
  return r.l == 0.0f ? 0.0f : exp2f(r.mp - r.m - kLift - log2f(r.l));
}
__device__ __forceinline__ float row_lse(const RowStats& r) {
  return r.l == 0.0f ? -INFINITY : (r.m + log2f(r.l)) * 0.6931471805599453f;
}

// Four columns of a finished row.
template <bool HALF>
__device__ __forceinline__ void store4(uint16_t* p, float4 v, float f) {
  uint2 o;
  if (f == 0.0f) {  // a row that saw nothing: its sums are 0 too
    o = make_uint2(0, 0);
  } else if (HALF) {
    o.x = pack_f16x2(v.x * f, v.y * f);
    o.y = pack_f16x2(v.z * f, v.w * f);
  } else {
    o.x = pack_bf16x2(v.x * f, v.y * f);
    o.y = pack_bf16x2(v.z * f, v.w * f);
  }
  *reinterpret_cast<uint2*>(p) = o;
}

// Where row `i` of tile `tile` (of cache head h) of sequence s reads and writes.
struct Row {
  int64_t token;
  int32_t head;
  bool there;
};
__device__ __forceinline__ Row row_of(const AttendArgs& a, int s, int64_t tile, int h, int rows, int i) {
  const int64_t c0 = __ldg(a.cu + s), c1 = __ldg(a.cu + s + 1);
  const uint32_t r = (uint32_t)(tile * rows + i), t = r / (uint32_t)a.group;  // below tokens * heads < 2^31
  Row w;
  w.token = c0 + t;
  w.head = h * a.group + (int)(r - t * (uint32_t)a.group);
  w.there = w.token < c1 && w.token >= 0 && w.token < a.tokens;
  return w;
}

template <int D, bool HALF>
__device__ __forceinline__ void write_row(const AttendArgs& a, const Row& w, int c, const RowStats& r,
                                          float4 o) {
  if (!w.there) return;
  const int64_t at = w.token * a.heads + w.head;
  store4<HALF>(a.out + at * D + c, o, out_factor(r));
  if (c == 0 && a.lse) a.lse[at] = row_lse(r);
}

// Items that several workers share are listed in the workspace behind the
// workers' slots (two each): the worker that an item begins with leaves the
// number of workers (0: its last item was finished) and where the item lies.
struct Shared {
  int32_t parts, s, tile, h;
};
template <int ROWS, int D>
__device__ __forceinline__ Shared* shared_items(const AttendArgs& a, int workers) {
  return reinterpret_cast<Shared*>(a.ws + (int64_t)workers * 2 * ROWS * (D + 4));
}

// Adds parts [i0, i1) of a shared item to (r, o), BATCH parts' loads at a time.
template <int BATCH, int ROWS, int D>
__device__ __forceinline__ void add_parts(const float* first, const float* rest, int i0, int i1, int at, int row,
                                          RowStats& r, float4& o) {
  constexpr int SLOT = ROWS * (D + 4);
  for (int i = i0; i < i1; i += BATCH) {
    float4 st[BATCH], x[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      st[k] = make_float4(kNone, kNone, 0.0f, 0.0f);
      x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i + k < i1) {
        const float* p = i + k == 0 ? first : rest + (int64_t)(i + k) * 2 * SLOT;
        st[k] = __ldg(reinterpret_cast<const float4*>(p + ROWS * D + row * 4));
        x[k] = __ldg(reinterpret_cast<const float4*>(p + at));
      }
    }
    float m = r.m, mp = r.mp;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      m = fmaxf(m, st[k].x);
      mp = fmaxf(mp, st[k].y);
    }
    r.l *= exp2f(r.m - m);
    float f = exp2f(r.mp - mp);
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      r.l += st[k].z * exp2f(st[k].x - m);
      f = exp2f(st[k].y - mp);
      o.x = fmaf(x[k].x, f, o.x);
      o.y = fmaf(x[k].y, f, o.y);
      o.z = fmaf(x[k].z, f, o.z);
      o.w = fmaf(x[k].w, f, o.w);
    }
    r.m = m;
    r.mp = mp;
  }
}

// Joins the shared items (64 sequences' tiles of 64 x 512 sums in 14 us, one in 152
// parts in 8; 32 sequences' of 8 x 128 in 5): every CTA reads the list, and all pieces of all items
// are spread over the grid. An item of few parts (a batch: two or three) is
// streamed, four columns a thread. Of a long one (a sequence alone on the GPU
// has up to 152 parts) sixteen threads take a sixteenth of the parts each, and are
// added up in order (four: 13 us).
template <int D, int ROWS, bool HALF>
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendArgs a, int workers) {
  constexpr int SLOT = ROWS * (D + 4), QUADS = ROWS * D / 4, FEW = 12;
  __shared__ int32_t list[512], start[513];
  __shared__ float4 sum[16][16];
  __shared__ float4 stat[16][16];
  grid_dependency_wait();
  allow_dependent_launch();
  const Shared* items = shared_items<ROWS, D>(a, workers);
  __shared__ int2 sums[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The list in the workers' order, and each item's first piece: two workers a thread.
  int parts[2];
  int2 before = make_int2(0, 0);  // items and pieces up to this thread's last
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int w = threadIdx.x * 2 + k;
    parts[k] = w < workers ? __ldg(&items[w].parts) : 0;
    before.x += parts[k] > 0;
    before.y += parts[k] > FEW ? QUADS / 16 : parts[k] > 0 ? (QUADS + 255) / 256 : 0;
  }
  const int2 mine = before;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, before.x, o), y = __shfl_up_sync(0xFFFFFFFFu, before.y, o);
    if (lane >= o) {
      before.x += x;
      before.y += y;
    }
  }
  if (lane == 31) sums[warp] = before;
  __syncthreads();
  int n = 0, total = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) {
    if (k < warp) {
      before.x += sums[k].x;
      before.y += sums[k].y;
    }
    n += sums[k].x;
    total += sums[k].y;
  }
  int at_item = before.x - mine.x, at_piece = before.y - mine.y;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (parts[k] > 0) {
      list[at_item] = threadIdx.x * 2 + k;
      start[at_item++] = at_piece;
      at_piece += parts[k] > FEW ? QUADS / 16 : (QUADS + 255) / 256;
    }
  __syncthreads();
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int lo = 0, hi = n;  // the item that piece u belongs to
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    const int w = list[lo], piece = u - start[lo];
    const Shared item = items[w];
    const float* first = a.ws + ((int64_t)w * 2 + 1) * SLOT;  // the worker's slot 1, then slots 0
    const float* rest = a.ws + (int64_t)w * 2 * SLOT;
    RowStats r = {kNone, kNone, 0.0f};
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (item.parts <= FEW) {
      const int at = (piece * 256 + threadIdx.x) * 4, row = at / D;
      if (at >= ROWS * D) continue;
      add_parts<4, ROWS, D>(first, rest, 0, item.parts, at, row, r, o);
      write_row<D, HALF>(a, row_of(a, item.s, item.tile, item.h, ROWS, row), at % D, r, o);
      continue;
    }
    const int v = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int at = (piece * 16 + v) * 4, row = at / D;
    const int each = (item.parts + 15) / 16, i0 = share * each, i1 = min(i0 + each, item.parts);
    add_parts<5, ROWS, D>(first, rest, i0, i1, at, row, r, o);
    __syncthreads();
    sum[share][v] = o;
    stat[share][v] = make_float4(r.m, r.mp, r.l, 0.0f);
    __syncthreads();
    if (share == 0) {
      for (int k = 1; k < 16; ++k) {
        const float4 st = stat[k][v], x = sum[k][v];
        const float m = fmaxf(r.m, st.x), mp = fmaxf(r.mp, st.y);
        r.l = r.l * exp2f(r.m - m) + st.z * exp2f(st.x - m);
        const float f0 = exp2f(r.mp - mp), f1 = exp2f(st.y - mp);
        o.x = o.x * f0 + x.x * f1;
        o.y = o.y * f0 + x.y * f1;
        o.z = o.z * f0 + x.z * f1;
        o.w = o.w * f0 + x.w * f1;
        r.m = m;
        r.mp = mp;
      }
      write_row<D, HALF>(a, row_of(a, item.s, item.tile, item.h, ROWS, row), at % D, r, o);
    }
  }
}

// The joining kernel behind a main kernel of `workers` CTAs.
template <int D, int ROWS, bool HALF>
cudaError_t launch_join(const AttendArgs& a, int workers, cudaStream_t stream) {
  return launch_dependent(attend_join_kernel<D, ROWS, HALF>, dim3(152 * 6), dim3(kThreads), 0, stream, a,
                          workers);
}

// Workspace of a main kernel of `workers` CTAs.
template <int D, int ROWS>
size_t join_bytes(int workers) {
  return (size_t)workers * (2 * ROWS * (D + 4) * sizeof(float) + sizeof(Shared));
}

}  // namespace

}  // namespace csa
