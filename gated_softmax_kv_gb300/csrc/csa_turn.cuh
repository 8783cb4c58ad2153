// Shared by the kernels that turn column pairs (csa_rope.cu, csa_norm_rope.cu):
// element types, 16-byte vectors, the angle of a position and the position of a
// compressed row. Not installed, not part of the ABI.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_device.cuh"

namespace csa {

struct Bf16 {
  uint16_t bits;
};

template <typename T>
struct Elem;
template <>
struct Elem<Bf16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(bf16_lo(w), bf16_hi(w));
  }
  static __device__ __forceinline__ uint32_t pack(float2 v) { return pack_bf16x2(v.x, v.y); }
  static __device__ __forceinline__ float load(const Bf16* p) {
    return __uint_as_float((uint32_t)p->bits << 16);
  }
  static __device__ __forceinline__ void store(Bf16* p, float v) {
    p->bits = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float2 v) {
    __half2 h = __float22half2_rn(v);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void store(__half* p, float v) { *p = __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};

// 16 bytes of T as fp32 values and back.
template <typename T>
struct Vec {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 w, float* v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<T>::unpack(u[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = Elem<T>::pack(make_float2(v[2 * i], v[2 * i + 1]));
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 w, float* v) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

// f / (2 pi) modulo 1 as a 64-bit fraction, from the bits of f: with f =
// m 2^(e-52), m a 53-bit integer, and K = floor(2^66 / (2 pi)), the product's
// high word (m 2^11) K / 2^64 times 2^(e-1) is 2^64 f / (2 pi). K lacks less than
// 2^-63 of itself and the high word, at least 2^62.3, less than one: together
// below 2^-61 relative, f 2^-61 / (2 pi) turns. A shift to the right drops less
// than 2^-64 turns, one to the left (f >= 4) or none (f >= 2) nothing.
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t b = (uint64_t)__double_as_longlong(f);
  const int e = (int)((b >> 52) & 0x7FF) - 1023;
  const uint64_t m = (b & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const uint64_t kInv2Pi = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi))
  const uint64_t p = __umul64hi(m << 11, kInv2Pi);
  const int s = e - 1;
  const uint64_t r = s <= -64 ? 0ull : s < 0 ? (p >> -s) : s < 64 ? (p << s) : 0ull;
  return (int64_t)b < 0 ? 0ull - r : r;
}

__device__ __forceinline__ void turn_of(uint64_t f, int64_t pos, float amplitude, float sign,
                                        float* c, float* s) {
  const uint64_t phase = f * (uint64_t)pos + 0x80000000ull;  // nearest of the top 32 bits
  const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
  float sn, cs;
  sincospif(half_turns, &sn, &cs);
  *c = cs * amplitude;
  *s = sn * (amplitude * sign);
}

// The position of token t. A: positions, position_bits, cu, nseq, search (the largest
// power of two below nseq, 0 for one segment) and ratio.
template <class A>
__device__ __forceinline__ int64_t position_of(const A& a, int64_t t) {
  if (a.positions)
    return a.position_bits == 64 ? __ldg(static_cast<const long long*>(a.positions) + t)
                                 : (int64_t)__ldg(static_cast<const int32_t*>(a.positions) + t);
  // the last s with cu[s] <= t, by halving steps of the same number for every
  // row, so that several rows' searches run side by side
  int lo = 0;
  int64_t base = __ldg(a.cu);
  for (int step = a.search; step; step >>= 1) {
    const int mid = lo + step;
    if (mid < a.nseq) {
      const int64_t at = __ldg(a.cu + mid);
      if (at <= t) {
        lo = mid;
        base = at;
      }
    }
  }
  return t >= __ldg(a.cu + a.nseq) ? 0 : (t - base) * a.ratio;
}

}  // namespace csa
