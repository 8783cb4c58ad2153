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

// Joins n partial results of one tile, each `ROWS` x D sums and the rows'
// statistics, in their order: part(i) gives the sums, stats(i) the statistics
// of part i.
template <int D, int ROWS, bool HALF, class Part, class Out>
__device__ __forceinline__ void join(int n, Part part, Out out) {
  for (int u = threadIdx.x; u < ROWS * (D / 4); u += kThreads) {
    const int row = u / (D / 4), c = (u % (D / 4)) * 4;
    RowStats r = {kNone, kNone, 0.0f};
    for (int i = 0; i < n; ++i) {
      const float* st = part(i) + ROWS * D + row * 4;
      r.m = fmaxf(r.m, st[0]);
      r.mp = fmaxf(r.mp, st[1]);
    }
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < n; ++i) {
      const float* p = part(i);
      const float* st = p + ROWS * D + row * 4;
      const float4 v = *reinterpret_cast<const float4*>(p + row * D + c);
      r.l += st[2] * exp2f(st[0] - r.m);
      const float f = exp2f(st[1] - r.mp);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    out(row, c, r, o);
  }
}

// Where row `i` of tile `tile` (of cache head h) of sequence s reads and writes.
struct Row {
  int64_t token;
  int32_t head;
  bool there;
};
__device__ __forceinline__ Row row_of(const AttendArgs& a, int s, int64_t tile, int h, int rows, int i) {
  const int64_t c0 = __ldg(a.cu + s), c1 = __ldg(a.cu + s + 1);
  const int64_t r = tile * rows + i, t = r / a.group;
  Row w;
  w.token = c0 + t;
  w.head = h * a.group + (int)(r - t * a.group);
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

// One CTA for each stretch's end: the first one inside an item joins it.
template <int D, int ROWS, bool HALF>
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendArgs a, const PlanShape plan) {
  __shared__ int64_t sums[kThreads / 32 + 1];
  __shared__ Place found;
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t w = (int64_t)blockIdx.x + 1;
  const Place place = locate<kThreads>(a, plan, w, sums, &found);
  if (place.pos < 0) return;
  const SeqWork work = seq_work(a, plan, place.s);
  const int64_t item = place.within / work.chunks;
  const int64_t c0 = place.within - item * work.chunks;
  if (c0 == 0 || c0 > place.per) return;  // between items, or an earlier end is inside this one
  const int h = (int)(item / work.tiles);
  const int64_t tile = item - h * work.tiles;
  const int n = 1 + (int)((work.chunks - c0 + place.per - 1) / place.per);
  constexpr int SLOT = ROWS * (D + 4);
  const float* ws = a.ws;
  join<D, ROWS, HALF>(
      n, [&](int i) { return ws + ((w - 1 + i) * 2 + (i == 0)) * SLOT; },
      [&](int row, int c, const RowStats& r, float4 v) {
        write_row<D, HALF>(a, row_of(a, place.s, tile, h, ROWS, row), c, r, v);
      });
}

}  // namespace

}  // namespace csa
