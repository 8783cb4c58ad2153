// Rotary positions (declared in include/csa_rope.h): turns column pairs of
// every head by position * frequency, in one pass over the data.
//
// Angles. A frequency f (radians a position, fp64) becomes F = f / (2 pi) in
// 64-bit fixed point, so the phase of position p is p * F modulo 2^64: the
// reduction to one turn is the integer product's own overflow, exact for any
// position, with no fp64 arithmetic per element (fp64 runs at 1/64 of the
// fp32 rate here). What is off is F, by turns_of's rounding, times p. The top
// 32 bits go through sincospif.
//
// The kernels are copies with some arithmetic, bound by memory. A thread keeps
// its columns for its whole loop, so F is worked out once per thread. 66533 rows
// of 512 bf16 columns, 64 of them turned, take 22 us (6.2 TB/s, 92% of the
// copy rate); 32768 tokens of 8 fp16 heads of 128 columns, all turned, 26.5 us
// (75%). A decoding step (16 tokens of 64 heads) takes 4 us, a launch's latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_device.cuh"
#include "csa_internal.h"
#include "csa_rope.h"
#include "csa_turn.cuh"

namespace csa {

namespace {

struct RopeArgs {
  const void* x;
  void* y;
  const double* freqs;
  const void* positions;
  const int32_t* cu;
  int64_t tokens;
  int64_t xt, xh, yt, yh;  // strides in elements
  int32_t position_bits, nseq, ratio;
  int32_t search;  // the largest power of two below nseq (0: one segment)
  int32_t heads, d, rope, offset;
  float amplitude;
  bool transpose, in_place;
};

// One pair of a head, as it lies in memory: next to one another or half a part
// apart.
template <typename E, bool HALF>
__device__ __forceinline__ void load_pair(const E* p, int half, uint32_t& a, uint32_t& b) {
  if constexpr (sizeof(E) == 4) {
    if constexpr (HALF) {
      a = __float_as_uint(p[0]);
      b = __float_as_uint(p[half]);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      a = v.x;
      b = v.y;
    }
  } else if constexpr (HALF) {
    a = reinterpret_cast<const uint16_t*>(p)[0];
    b = reinterpret_cast<const uint16_t*>(p)[half];
  } else {
    a = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <typename E, bool HALF>
__device__ __forceinline__ float2 pair_value(uint32_t a, uint32_t b) {
  if constexpr (sizeof(E) == 4)
    return make_float2(__uint_as_float(a), __uint_as_float(b));
  else
    return Elem<E>::unpack(HALF ? a | (b << 16) : a);
}
template <typename E, bool HALF>
__device__ __forceinline__ void store_pair(E* p, int half, float2 v) {
  if constexpr (HALF) {
    Elem<E>::store(p, v.x);
    Elem<E>::store(p + half, v.y);
  } else if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float2*>(p) = v;
  } else {
    *reinterpret_cast<uint32_t*>(p) = Elem<E>::pack(v);
  }
}

// Vector kernel where heads share sines: 16-byte aligned rows, part and
// strides. A chunk is 16 bytes of interleaved pairs, twice 16 bytes half a part
// apart, or (out of place) one vector to copy; a thread has the same chunk of
// four heads of every token that it visits, and issues their loads before it
// works out the angles.
template <typename E, bool HALF>
__global__ void __launch_bounds__(256) rope_heads_kernel(const RopeArgs a, int32_t chunks, int32_t groups) {
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int N = Vec<E>::N, H = 4;
  constexpr int PAIRS = HALF ? N : N / 2;
  const uint32_t id = blockIdx.x * blockDim.x + threadIdx.x;
  const uint32_t lanes = gridDim.x * blockDim.x / chunks;  // whole rows of chunks
  const uint32_t first = id / chunks;
  const int c = (int)(id - first * chunks);
  if (first >= lanes) return;
  const int turned = a.rope / (2 * PAIRS);
  const bool turns = c < turned;
  const int k = (c - turned) * N;
  const int col = turns ? a.offset + c * N : k < a.offset ? k : k + a.rope;
  const int64_t items = a.tokens * groups;
  const E* x = static_cast<const E*>(a.x) + col;
  E* y = static_cast<E*>(a.y) + col;
  uint64_t f[PAIRS];
  if (turns) {
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) f[i] = turns_of(__ldg(a.freqs + c * PAIRS + i));
  }
  const float sign = a.transpose ? -1.0f : 1.0f;
  for (int64_t it = first; it < items; it += lanes) {
    const int64_t token = it / groups;
    const int head = (int)(it - token * groups) * H;
    uint4 v[H], w[H];
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (head + h < a.heads) {
        const E* p = x + token * a.xt + (head + h) * a.xh;
        v[h] = *reinterpret_cast<const uint4*>(p);
        if (HALF && turns) w[h] = *reinterpret_cast<const uint4*>(p + a.rope / 2);
      }
    if (turns) {
      const int64_t pos = position_of(a, token);
      float cs[PAIRS], sn[PAIRS];
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) turn_of(f[i], pos, a.amplitude, sign, &cs[i], &sn[i]);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float p[N];
        Vec<E>::unpack(v[h], p);
        if constexpr (HALF) {
          float q[N], va[N], wb[N];
          Vec<E>::unpack(w[h], q);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            va[i] = fmaf(-q[i], sn[i], p[i] * cs[i]);
            wb[i] = fmaf(p[i], sn[i], q[i] * cs[i]);
          }
          v[h] = Vec<E>::pack(va);
          w[h] = Vec<E>::pack(wb);
        } else {
          float o[N];
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            o[2 * i] = fmaf(-p[2 * i + 1], sn[i], p[2 * i] * cs[i]);
            o[2 * i + 1] = fmaf(p[2 * i], sn[i], p[2 * i + 1] * cs[i]);
          }
          v[h] = Vec<E>::pack(o);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (head + h < a.heads) {
        E* p = y + token * a.yt + (head + h) * a.yh;
        *reinterpret_cast<uint4*>(p) = v[h];
        if (HALF && turns) *reinterpret_cast<uint4*>(p + a.rope / 2) = w[h];
      }
  }
}

// The position of a token, worked out by a warp: segments are searched 32 at a
// time.
__device__ __forceinline__ int64_t warp_position(const RopeArgs& a, int64_t t, int lane) {
  if (a.positions) return position_of(a, t);
  int lo = 0, span = a.nseq;  // the segment is in [lo, lo + span)
  while (span > 1) {
    const int step = (span + 31) / 32, at = lo + lane * step;
    const bool before = lane * step < span && __ldg(a.cu + at) <= t;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, before);
    const int k = who ? 31 - __clz(who) : 0;
    span = min(step, span - k * step);
    lo += k * step;
  }
  return t >= __ldg(a.cu + a.nseq) ? 0 : (t - __ldg(a.cu + lo)) * a.ratio;
}

// Rows that share nothing (one head, or a decoding step): whole warps turn 32
// pairs of a row at a time, a lane a pair, so that a row's sines cost one pass of
// a warp; the other half of the CTA's warps copy what is not turned, 16 bytes a
// thread. One kernel whose lanes did either cost 455 instructions a warp and row
// of 512 bf16 columns, 64 of them turned (58 us for 66533 rows); this one about a
// third of that (22 us). Four rows a warp and thread at once measured the same
// there, and 20.5 us against 17.8 for rows of 128 columns.
template <typename E, bool HALF>
__global__ void __launch_bounds__(256) rope_rows_kernel(const RopeArgs a, int32_t blocks_of_pairs, int32_t copied) {
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int N = Vec<E>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = a.tokens * a.heads;
  const int turners = copied ? 4 : 8;  // warps of the CTA
  if (warp < turners) {
    const int64_t id = (int64_t)blockIdx.x * turners + warp, warps = (int64_t)gridDim.x * turners;
    // each warp keeps one block of pairs
    const int64_t each = warps / blocks_of_pairs;
    const int block = (int)(id / (each > 0 ? each : 1));
    if (each == 0 || block >= blocks_of_pairs) return;
    const int pair = block * 32 + lane, pairs = a.rope / 2;
    const bool on = pair < pairs;
    const uint64_t f = on ? turns_of(__ldg(a.freqs + pair)) : 0;
    const int col = a.offset + (HALF ? pair : 2 * pair);
    const E* x = static_cast<const E*>(a.x) + col;
    E* y = static_cast<E*>(a.y) + col;
    const float sign = a.transpose ? -1.0f : 1.0f;
    for (int64_t r = id - block * each; r < rows; r += each) {
      const int64_t token = a.heads == 1 ? r : r / a.heads;
      const int head = (int)(r - token * a.heads);
      uint32_t va, vb;
      if (on) load_pair<E, HALF>(x + token * a.xt + head * a.xh, pairs, va, vb);
      float c, s;
      turn_of(f, warp_position(a, token, lane), a.amplitude, sign, &c, &s);
      const float2 p = pair_value<E, HALF>(va, vb);
      if (on)
        store_pair<E, HALF>(y + token * a.yt + head * a.yh, pairs,
                            make_float2(fmaf(-p.y, s, p.x * c), fmaf(p.x, s, p.y * c)));
    }
  } else {
    const uint32_t id = blockIdx.x * 128 + threadIdx.x - 128, lanes = gridDim.x * 128 / copied;
    const uint32_t first = id / copied;
    const int c = (int)(id - first * copied) * N;
    if (first >= lanes) return;
    const int col = c < a.offset ? c : c + a.rope;
    const E* x = static_cast<const E*>(a.x) + col;
    E* y = static_cast<E*>(a.y) + col;
    for (int64_t r = first; r < rows; r += lanes) {
      const int64_t token = a.heads == 1 ? r : r / a.heads;
      const int head = (int)(r - token * a.heads);
      *reinterpret_cast<uint4*>(y + token * a.yt + head * a.yh) =
          ld_stream(reinterpret_cast<const uint16_t*>(x + token * a.xt + head * a.xh));
    }
  }
}

// Any alignment, any even part: a thread takes one pair or one column.
template <typename T, bool HALF>
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int pairs = a.rope / 2;
  const int units = pairs + (a.in_place ? 0 : a.d - a.rope);
  const int64_t items = a.tokens * a.heads * units;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  for (int64_t it = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; it < items;
       it += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = it / units;
    const int u = (int)(it - row * units);
    const int64_t t = row / a.heads;
    const int h = (int)(row - t * a.heads);
    const T* px = x + t * a.xt + h * a.xh;
    T* py = y + t * a.yt + h * a.yh;
    if (u < pairs) {
      float c, s;
      turn_of(turns_of(__ldg(a.freqs + u)), position_of(a, t), a.amplitude,
              a.transpose ? -1.0f : 1.0f, &c, &s);
      const int ia = a.offset + (HALF ? u : 2 * u), ib = HALF ? ia + pairs : ia + 1;
      const float va = Elem<T>::load(px + ia), vb = Elem<T>::load(px + ib);
      Elem<T>::store(py + ia, fmaf(-vb, s, va * c));
      Elem<T>::store(py + ib, fmaf(va, s, vb * c));
    } else {
      const int k = u - pairs;
      const int col = k < a.offset ? k : k + a.rope;
      py[col] = px[col];
    }
  }
}

template <typename T, bool HALF>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  const uintptr_t bytes = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
  const int64_t cols = a.xt | a.xh | a.yt | a.yh | a.offset | a.d | (HALF ? a.rope / 2 : a.rope);
  if (bytes % 16 == 0 && cols % N == 0) {
    constexpr int WIDE = HALF ? N : N / 2;
    const int copied = a.in_place ? 0 : (a.d - a.rope) / N;
    // Heads share a token's sines, four at a time, where the rows' turned pairs are
    // enough work for that (in warps of 32 pairs). Measured as a graph, rows kernel
    // against this: 8 heads of 128 fp16 columns, all turned, 256 tokens (4096 warps)
    // 2.9 us / 3.7, 512 tokens 4.3 / 3.7, 2048 tokens 8.2 / 3.9; 64 heads of 512, 64
    // turned, 16 tokens (1024) 2.2 / 2.7, 64 tokens (4096) 3.9 / 2.9; all of 512
    // turned, 16 tokens (8192) 4.2 / 2.8, 256 tokens 23.9 / 7.3.
    const int chunks = a.rope / (2 * WIDE) + copied, groups = (a.heads + 3) / 4;
    const int64_t most = 152 * 4;
    if (a.heads >= 4 && a.tokens * a.heads * ((a.rope / 2 + 31) / 32) >= 4096) {
      int64_t blocks = (a.tokens * groups * chunks + 255) / 256;
      if (blocks > most) blocks = most;
      const int64_t least = (chunks + 255) / 256;  // at least one whole row of chunks
      if (blocks < least) blocks = least;
      return launch_dependent(rope_heads_kernel<T, HALF>, dim3((unsigned)blocks), dim3(256), 0, stream, a,
                              (int32_t)chunks, (int32_t)groups);
    }
    const int64_t rows = a.tokens * a.heads;
    const int pairs32 = (a.rope / 2 + 31) / 32, turners = copied ? 4 : 8;
    int64_t blocks = (rows * pairs32 + turners - 1) / turners;
    const int64_t copies = (rows * copied + 127) / 128;
    if (blocks < copies) blocks = copies;
    if (blocks > 2 * most) blocks = 2 * most;
    const int64_t least = (pairs32 + turners - 1) / turners > (copied + 127) / 128
                              ? (pairs32 + turners - 1) / turners
                              : (copied + 127) / 128;  // every block of pairs, a whole row of copies
    if (blocks < least) blocks = least;
    return launch_dependent(rope_rows_kernel<T, HALF>, dim3((unsigned)blocks), dim3(256), 0, stream, a,
                            (int32_t)pairs32, (int32_t)copied);
  }
  const int64_t items = a.tokens * a.heads * (a.rope / 2 + (a.in_place ? 0 : a.d - a.rope));
  int64_t blocks = (items + 255) / 256;
  if (blocks > 152 * 32) blocks = 152 * 32;
  return launch_dependent(rope_any_kernel<T, HALF>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

template <typename T>
cudaError_t launch_rope_layout(const RopeArgs& a, int32_t layout, cudaStream_t stream) {
  return layout == CSA_ROPE_HALF ? launch_rope<T, true>(a, stream) : launch_rope<T, false>(a, stream);
}

}  // namespace

}  // namespace csa

extern "C" csa_status_t csa_rope(const void* x, void* y, const double* freqs, const void* positions,
                                 int32_t position_bits, const int32_t* cu_rows, int32_t num_seqs,
                                 int32_t ratio, int64_t tokens, int32_t heads, int32_t head_dim,
                                 int64_t x_token_stride, int64_t x_head_stride,
                                 int64_t y_token_stride, int64_t y_head_stride, int32_t rope_dim,
                                 int32_t offset, int32_t layout, int32_t dtype, float amplitude,
                                 int32_t transpose, cudaStream_t stream) {
  if (dtype != CSA_BF16 && dtype != CSA_FP16 && dtype != CSA_FP32) return CSA_ERR_UNSUPPORTED;
  if (layout != CSA_ROPE_INTERLEAVED && layout != CSA_ROPE_HALF) return CSA_ERR_UNSUPPORTED;
  if (rope_dim < 2 || rope_dim % 2 != 0 || offset < 0 || head_dim < 1 ||
      (int64_t)offset + rope_dim > head_dim)
    return CSA_ERR_UNSUPPORTED;
  if (positions && position_bits != 32 && position_bits != 64) return CSA_ERR_UNSUPPORTED;
  if (tokens < 0 || heads < 1) return CSA_ERR_RANGE;
  if (x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0)
    return CSA_ERR_RANGE;
  // no index may pass 63 bits
  const int64_t most = (int64_t)1 << 60;
  if (tokens > most / heads / head_dim) return CSA_ERR_RANGE;
  const int64_t by_token = tokens > 1 ? most / (tokens - 1) : most;
  const int64_t by_head = heads > 1 ? most / (heads - 1) : most;
  if (x_token_stride > by_token || y_token_stride > by_token || x_head_stride > by_head ||
      y_head_stride > by_head)
    return CSA_ERR_RANGE;
  // distinct output elements: heads within a token's stretch, or tokens within a head's
  const int64_t head_span = (heads - 1) * y_head_stride + head_dim;
  const int64_t token_span = tokens > 0 ? (tokens - 1) * y_token_stride + head_dim : 0;
  const bool heads_apart = heads == 1 || y_head_stride >= head_dim;
  const bool tokens_apart = tokens <= 1 || y_token_stride >= head_dim;
  if (!heads_apart || !tokens_apart) return CSA_ERR_RANGE;
  if (heads > 1 && tokens > 1 && y_token_stride < head_span && y_head_stride < token_span)
    return CSA_ERR_RANGE;
  if (!freqs || (!positions && !cu_rows)) return CSA_ERR_NULL;
  if (!positions && (num_seqs < 1 || ratio < 1)) return CSA_ERR_RANGE;
  if (tokens > 0 && (!x || !y)) return CSA_ERR_NULL;
  const uintptr_t size = dtype == CSA_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % size != 0 ||
      reinterpret_cast<uintptr_t>(freqs) % 8 != 0 || reinterpret_cast<uintptr_t>(cu_rows) % 4 != 0 ||
      (positions && reinterpret_cast<uintptr_t>(positions) % (position_bits / 8) != 0))
    return CSA_ERR_ALIGN;
  const bool same = x == y;
  if (same && ((tokens > 1 && x_token_stride != y_token_stride) ||
               (heads > 1 && x_head_stride != y_head_stride)))
    return CSA_ERR_RANGE;
  if (tokens == 0) return CSA_OK;
  csa::RopeArgs a;
  a.x = x;
  a.y = y;
  a.freqs = freqs;
  a.positions = positions;
  a.cu = cu_rows;
  a.tokens = tokens;
  a.xt = tokens > 1 ? x_token_stride : 0;  // the stride of a single element is never stepped
  a.xh = heads > 1 ? x_head_stride : 0;
  a.yt = tokens > 1 ? y_token_stride : 0;
  a.yh = heads > 1 ? y_head_stride : 0;
  a.position_bits = position_bits;
  a.nseq = num_seqs;
  a.ratio = ratio;
  a.search = 0;
  for (int64_t step = 1; !positions && step < num_seqs; step *= 2) a.search = (int32_t)step;
  a.heads = heads;
  a.d = head_dim;
  a.rope = rope_dim;
  a.offset = offset;
  a.amplitude = amplitude;
  a.transpose = transpose != 0;
  a.in_place = same;
  const cudaError_t e = dtype == CSA_BF16   ? csa::launch_rope_layout<csa::Bf16>(a, layout, stream)
                        : dtype == CSA_FP16 ? csa::launch_rope_layout<__half>(a, layout, stream)
                                            : csa::launch_rope_layout<float>(a, layout, stream);
  return e == cudaSuccess ? CSA_OK : csa::record_cuda_error(e);
}
