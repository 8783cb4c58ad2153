// Norms of queries and keys for each head with the rotary positions in the same
// pass, and their gradient (declared in include/csa_norm_rope.h).
//
// A group of G lanes (4 .. 32) owns a head: a lane holds K vectors of 16 bytes of
// it, so a mean over the head is log2(G) shuffles and each byte is read once. For
// the half layout a lane's vectors come in pairs half a part apart, so that both
// columns of a pair are its own. A group keeps its columns for its whole loop:
// weights are read once. The lanes share a token's sines through shared memory, and
// they serve a span of its heads, whose first loads are issued before the sines.
//
// The gradient reads x and grad once, works r out again, and sums its part of dw
// in registers over the loop; the groups' sums meet in shared memory in a fixed
// order, and a second kernel adds the CTAs' in theirs.
//
// Angles are those of csa_rope.cu. Memory bounds the forward, with instructions close: 32768
// tokens of 40 bf16 heads of 128 columns, half turned, 118 us (5.7 TB/s, 84% of the copy
// rate). The gradient holds x, the gradient and the weights' sums of a lane's columns, 96
// registers: 16384 tokens of 40 heads, all turned, 133 us (3.8 TB/s).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "csa_cache_internal.h"
#include "csa_device.cuh"
#include "csa_internal.h"
#include "csa_norm_rope.h"
#include "csa_turn.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxHeadDim = 1024;

struct Side {
  const void* x;
  const void* weight;
  const void* grad;
  void* y;
  void* dweight;
  int64_t xt, xh, gt, gh, yt, yh;
  int64_t items;   // tokens x groups of heads
  int32_t heads;
  int32_t span;    // heads of an item
  int32_t groups;  // items of a token
  int32_t blocks;  // CTAs of this side
};

struct NormArgs {
  Side side[2];
  const double* freqs;
  const void* positions;
  const int32_t* cu;
  float* partial;  // [blocks of both sides][d]
  int64_t tokens;
  int32_t position_bits, nseq, ratio, search;
  int32_t d, rope, offset;
  int32_t lanes;  // G
  bool weight32;
  float amplitude, eps;
};

// N values of E as they are loaded: 16 bytes, or for the half layout of 16-bit types 8,
// since a lane has two vectors of each pair (fewer registers: 16384 tokens of 40 heads of
// 128, forward 86 us, backward 154 with 16 bytes).
template <typename E, int N>
struct Chunk {
  using Raw = uint4;
  static __device__ __forceinline__ Raw none() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void unpack(Raw w, float2 (&v)[N / 2]) {
    if constexpr (sizeof(E) == 4) {
      v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
      v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    } else {
      v[0] = Elem<E>::unpack(w.x);
      v[1] = Elem<E>::unpack(w.y);
      v[2] = Elem<E>::unpack(w.z);
      v[3] = Elem<E>::unpack(w.w);
    }
  }
  static __device__ __forceinline__ Raw pack(const float2 (&v)[N / 2]) {
    if constexpr (sizeof(E) == 4)
      return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    else
      return make_uint4(Elem<E>::pack(v[0]), Elem<E>::pack(v[1]), Elem<E>::pack(v[2]), Elem<E>::pack(v[3]));
  }
};
template <typename E>
struct Chunk<E, sizeof(E) == 2 ? 4 : -1> {
  using Raw = uint2;
  static __device__ __forceinline__ Raw none() { return make_uint2(0, 0); }
  static __device__ __forceinline__ void unpack(Raw w, float2 (&v)[2]) {
    v[0] = Elem<E>::unpack(w.x);
    v[1] = Elem<E>::unpack(w.y);
  }
  static __device__ __forceinline__ Raw pack(const float2 (&v)[2]) { return make_uint2(Elem<E>::pack(v[0]), Elem<E>::pack(v[1])); }
};
template <typename E, bool HALF>
constexpr int kChunk = HALF && sizeof(E) == 2 ? 4 : Vec<E>::N;

template <typename E>
__device__ __forceinline__ float weight_at(const NormArgs& a, const Side& s, int c) {
  return a.weight32 ? __ldg(static_cast<const float*>(s.weight) + c) : Elem<E>::load(static_cast<const E*>(s.weight) + c);
}

// Sum over the G = 4 .. 32 lanes of a group, the same in each.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes > 16) v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
  if (lanes > 8) v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
  if (lanes > 4) v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 1);
}

// Which columns a lane has: col[k] of its vector k, -1 for none; its first pair of
// turned columns, -1 where the vector is only normed.
template <int N, int K, bool HALF>
__device__ __forceinline__ void columns_of(const NormArgs& a, int lane, int (&col)[K], int (&pair)[K]) {
  const int first = a.offset / N, total = a.d / N;
  if constexpr (HALF) {
    static_assert(K % 2 == 0, "vectors in pairs");
    const int hp = a.rope / (2 * N);
#pragma unroll
    for (int k = 0; k < K; k += 2) {
      const int p = lane + a.lanes * (k / 2);
      if (p < hp) {
        col[k] = (first + p) * N;
        col[k + 1] = (first + hp + p) * N;
        pair[k] = pair[k + 1] = p * N;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = 2 * (p - hp) + i;  // of the vectors that are not turned
          const int v = u < first ? u : u + 2 * hp;
          col[k + i] = v < total ? v * N : -1;
          pair[k + i] = -1;
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = lane + a.lanes * k;
      col[k] = v < total ? v * N : -1;
      pair[k] = v < total && v >= first && v < first + a.rope / N ? (v - first) * (N / 2) : -1;
    }
  }
}

// The turn of a group's vectors, or its transpose: vectors 2j and 2j + 1 are the two
// halves of the same pairs, or a vector has whole pairs. Sines are those of the vector's
// N / 2 pairs, or of the first and second half of the N pairs of two vectors.
template <int N, int K, bool HALF, bool TRANSPOSE>
__device__ __forceinline__ void turn_vectors(float2 (&v)[K][N / 2], const int (&pair)[K], const float (&cs)[K][N / 2],
                                             const float (&sn)[K][N / 2]) {
  if constexpr (HALF) {
#pragma unroll
    for (int k = 0; k < K; k += 2)
      if (pair[k] >= 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const int h = k + 2 * i / (N / 2), j = 2 * i % (N / 2);
          const float2 c = make_float2(cs[h][j], cs[h][j + 1]);
          const float2 s = TRANSPOSE ? make_float2(-sn[h][j], -sn[h][j + 1]) : make_float2(sn[h][j], sn[h][j + 1]);
          const float2 n = make_float2(-s.x, -s.y), x = v[k][i], y = v[k + 1][i];
          v[k][i] = fma2_rn(y, n, mul2_rn(x, c));
          v[k + 1][i] = fma2_rn(x, s, mul2_rn(y, c));
        }
      }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (pair[k] >= 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float c = cs[k][i], s = TRANSPOSE ? -sn[k][i] : sn[k][i];
          const float2 x = v[k][i];
          v[k][i] = make_float2(fmaf(-x.y, s, x.x * c), fmaf(x.x, s, x.y * c));
        }
      }
  }
}

// The last segment that begins at or before token t, by the 32 lanes of a group that is
// a warp: two dependent loads for up to 1024 segments.
__device__ __forceinline__ int64_t warp_position_of(const NormArgs& a, int64_t t, int lane) {
  if (a.positions) return position_of(a, t);
  int lo = 0, span = a.nseq;
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

// H: heads that a group has in flight; an item is a token and a.span of a side's heads.
// Five CTAs an SM for the gradient of eight columns a lane (96 registers): 142 us, so 133.
// No number for the others: with one, 1 already, the compiler takes 112 registers for the
// forward instead of 72 to 88 (32768 tokens of 40 heads of 128, half turned: 152 us instead of 118).
template <typename E, int K, int H, bool HALF, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD && K * kChunk<E, HALF> <= 8 ? 5 : 0) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = kChunk<E, HALF>;
  using V = Chunk<E, N>;
  using Raw = typename V::Raw;
  // frequencies in turns, then each group's sines of its token
  extern __shared__ __align__(16) uint64_t freq[];
  __shared__ float sums[BWD ? kMaxHeadDim : 1];
  grid_dependency_wait();
  allow_dependent_launch();
  const bool second = (int)blockIdx.x >= a.side[0].blocks;
  const Side& s = a.side[second];
  const int block = (int)blockIdx.x - (second ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & (a.lanes - 1), group = threadIdx.x / a.lanes, groups = kThreads / a.lanes;
  const int pairs = a.rope / 2;
  float2* const turns = reinterpret_cast<float2*>(freq + ((pairs + 1) & ~1)) + group * pairs;
  for (int i = threadIdx.x; i < pairs; i += kThreads) freq[i] = turns_of(__ldg(a.freqs + i));
  int col[K], pair[K];
  columns_of<N, K, HALF>(a, lane, col, pair);
  float2 w[K][N / 2];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      w[k][i] = col[k] >= 0 ? make_float2(weight_at<E>(a, s, col[k] + 2 * i), weight_at<E>(a, s, col[k] + 2 * i + 1))
                            : make_float2(0.0f, 0.0f);
  float2 dw[BWD ? K : 1][N / 2];
#pragma unroll
  for (int k = 0; k < (BWD ? K : 1); ++k)
#pragma unroll
    for (int i = 0; i < N / 2; ++i) dw[k][i] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const float inv_d = 1.0f / (float)a.d;
  const int64_t step = (int64_t)s.blocks * groups;
  const int batches = (s.span + H - 1) / H;
  // every group of a warp makes the same number of rounds: shuffles need all lanes
  const int64_t rounds = (s.items + step - 1) / step;
  for (int64_t n = 0; n < rounds; ++n) {
    const int64_t it = n * step + (int64_t)block * groups + group;
    const bool on = it < s.items;
    const int64_t token = on ? it / s.groups : 0;
    const int first = on ? (int)(it - token * s.groups) * s.span : 0;
    const int heads = on ? min(s.span, s.heads - first) : 0;
    const E* const x0 = static_cast<const E*>(s.x) + token * s.xt + first * s.xh;
    const E* const g0 = BWD ? static_cast<const E*>(s.grad) + token * s.gt + first * s.gh : nullptr;
    E* const y0 = static_cast<E*>(s.y) + token * s.yt + first * s.yh;
    Raw xr[H][K], gr[BWD ? H : 1][K];
    auto load = [&](int h0) {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const bool there = h0 + h < heads && col[k] >= 0;
          xr[h][k] = there ? *reinterpret_cast<const Raw*>(x0 + (h0 + h) * s.xh + col[k]) : V::none();
          if constexpr (BWD)
            gr[h][k] = there ? *reinterpret_cast<const Raw*>(g0 + (h0 + h) * s.gh + col[k]) : V::none();
        }
    };
    load(0);
    // the token's sines, a pair a lane at a time, for all of its heads
    const int64_t pos = a.lanes == 32 ? warp_position_of(a, token, lane) : position_of(a, token);
    __syncwarp();
    for (int i = lane; i < pairs; i += a.lanes) {
      float2 t;
      turn_of(freq[i], pos, a.amplitude, 1.0f, &t.x, &t.y);
      turns[i] = t;
    }
    __syncwarp();
    float cs[K][N / 2], sn[K][N / 2];
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (pair[k] >= 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 t = turns[pair[k] + (HALF ? (k & 1) * (N / 2) : 0) + i];
          cs[k][i] = t.x;
          sn[k][i] = t.y;
        }
      }
#pragma unroll 1
    for (int b = 0; b < batches; ++b) {
      if (b > 0) load(b * H);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float2 x[K][N / 2], sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          V::unpack(xr[h][k], x[k]);
#pragma unroll
          for (int i = 0; i < N / 2; ++i) sum = fma2_rn(x[k][i], x[k][i], sum);
        }
        // rsqrtf is within 2 ulp
        const float r = rsqrtf(fmaf(group_sum(sum.x + sum.y, a.lanes), inv_d, a.eps));
        const float2 r2 = make_float2(r, r);
        const bool there = b * H + h < heads;
        if constexpr (!BWD) {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) x[k][i] = mul2_rn(mul2_rn(x[k][i], r2), w[k][i]);
          turn_vectors<N, K, HALF, false>(x, pair, cs, sn);
        } else {
          float2 g[K][N / 2], along = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < K; ++k) V::unpack(gr[h][k], g[k]);
          turn_vectors<N, K, HALF, true>(g, pair, cs, sn);
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
              if (there) dw[k][i] = fma2_rn(g[k][i], mul2_rn(x[k][i], r2), dw[k][i]);
              g[k][i] = mul2_rn(g[k][i], w[k][i]);
              along = fma2_rn(g[k][i], x[k][i], along);
            }
          const float back = -group_sum(along.x + along.y, a.lanes) * inv_d * r * r;
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) x[k][i] = mul2_rn(r2, fma2_rn(x[k][i], make_float2(back, back), g[k][i]));
        }
        if (there) {
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (col[k] >= 0) *reinterpret_cast<Raw*>(y0 + (b * H + h) * s.yh + col[k]) = V::pack(x[k]);
        }
      }
    }
  }
  if constexpr (BWD) {  // the CTA's sums: group by group
    for (int turn = 0; turn < groups; ++turn) {
      if (group == turn) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (col[k] >= 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float v = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x;
              sums[col[k] + i] = turn == 0 ? v : sums[col[k] + i] + v;
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.d; c += kThreads) a.partial[(int64_t)blockIdx.x * a.d + c] = sums[c];
  }
}

// Any alignment, any even part: a warp a head, a lane a pair or a column at a time;
// the gradient's sums in shared memory, a line a warp.
template <typename E, bool HALF, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const __grid_constant__ NormArgs a) {
  constexpr int WARPS = kThreads / 32;
  __shared__ float sums[BWD ? WARPS : 1][BWD ? kMaxHeadDim : 1];
  grid_dependency_wait();
  allow_dependent_launch();
  const bool second = (int)blockIdx.x >= a.side[0].blocks;
  const Side& s = a.side[second];
  const int block = (int)blockIdx.x - (second ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (BWD) {
    for (int c = lane; c < a.d; c += 32) sums[warp][c] = 0.0f;
    __syncwarp();
  }
  const int pairs = a.rope / 2, units = pairs + a.d - a.rope;
  const float inv_d = 1.0f / (float)a.d;
  for (int64_t it = (int64_t)block * WARPS + warp; it < s.items; it += (int64_t)s.blocks * WARPS) {
    const int64_t token = it / s.heads;
    const int head = (int)(it - token * s.heads);
    const E* x = static_cast<const E*>(s.x) + token * s.xt + head * s.xh;
    const E* g = static_cast<const E*>(s.grad) + token * s.gt + head * s.gh;
    E* y = static_cast<E*>(s.y) + token * s.yt + head * s.yh;
    float sum = 0.0f;
    for (int c = lane; c < a.d; c += 32) {
      const float v = Elem<E>::load(x + c);
      sum = fmaf(v, v, sum);
    }
    const float r = 1.0f / sqrtf(fmaf(group_sum(sum, 32), inv_d, a.eps));
    const int64_t pos = position_of(a, token);
    float back = 0.0f;
    // backward: a first round for mean(u x), a second for the gradient
    for (int round = BWD ? 0 : 1; round < 2; ++round) {
      float along = 0.0f;
      for (int u = lane; u < units; u += 32) {
        const bool turned = u < pairs;
        const int k = u - pairs;
        const int ca = turned ? a.offset + (HALF ? u : 2 * u) : k < a.offset ? k : k + a.rope;
        const int cb = turned ? (HALF ? ca + pairs : ca + 1) : ca;
        float c = 1.0f, sn = 0.0f;
        if (turned) turn_of(turns_of(__ldg(a.freqs + u)), pos, a.amplitude, 1.0f, &c, &sn);
        const float xa = Elem<E>::load(x + ca), xb = Elem<E>::load(x + cb);
        const float wa = weight_at<E>(a, s, ca), wb = weight_at<E>(a, s, cb);
        float oa, ob;
        if constexpr (!BWD) {
          const float na = xa * r * wa, nb = xb * r * wb;
          oa = turned ? fmaf(-nb, sn, na * c) : na;
          ob = fmaf(na, sn, nb * c);
        } else {
          const float ga = Elem<E>::load(g + ca), gb = Elem<E>::load(g + cb);
          const float ha = turned ? fmaf(gb, sn, ga * c) : ga, hb = fmaf(-ga, sn, gb * c);
          if (round == 0) {
            sums[warp][ca] = fmaf(ha, xa * r, sums[warp][ca]);
            along = fmaf(ha * wa, xa, along);
            if (turned) {
              sums[warp][cb] = fmaf(hb, xb * r, sums[warp][cb]);
              along = fmaf(hb * wb, xb, along);
            }
            continue;
          }
          oa = r * fmaf(-xa, back, ha * wa);
          ob = r * fmaf(-xb, back, hb * wb);
        }
        Elem<E>::store(y + ca, oa);
        if (turned) Elem<E>::store(y + cb, ob);
      }
      __syncwarp();
      if (BWD && round == 0) back = group_sum(along, 32) * inv_d * r * r;
    }
  }
  if constexpr (BWD) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) v += sums[k][c];
      a.partial[(int64_t)blockIdx.x * a.d + c] = v;
    }
  }
}

// dw of both sides from the CTAs' sums: 32 columns a CTA, 32 lines of CTAs summed
// apart and then in order (8 lines: 10 us for 607 CTAs' sums of 128).
constexpr int kLines = 32;
template <typename E>
__global__ void __launch_bounds__(32 * kLines) norm_weights_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[kLines][32];
  grid_dependency_wait();
  allow_dependent_launch();
  const Side& s = a.side[blockIdx.y];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), line = threadIdx.x >> 5;
  const float* p = a.partial + (int64_t)(blockIdx.y ? a.side[0].blocks : 0) * a.d;
  float v = 0.0f;
  if (c < a.d) {
#pragma unroll 8
    for (int b = line; b < s.blocks; b += kLines) v += p[(int64_t)b * a.d + c];
  }
  part[line][threadIdx.x & 31] = v;
  __syncthreads();
  if (line == 0 && c < a.d) {
#pragma unroll
    for (int k = 1; k < kLines; ++k) v += part[k][threadIdx.x];
    if (a.weight32)
      static_cast<float*>(s.dweight)[c] = v;
    else
      Elem<E>::store(static_cast<E*>(s.dweight) + c, v);
  }
}

// CTAs of the two sides: as many as there is work for, at most `most` together,
// shared in proportion to their heads.
void deal_out(NormArgs& a, int64_t per_block, int64_t most) {
  int64_t want[2];
  for (int k = 0; k < 2; ++k) want[k] = (a.side[k].items + per_block - 1) / per_block;
  const bool many = want[0] + want[1] > most;
  const int64_t heads = a.side[0].heads + a.side[1].heads;
  for (int k = 0; k < 2; ++k) {
    int64_t b = want[k];
    const int64_t share = most * a.side[k].heads / heads;
    if (many && b > share) b = share;
    if (b < 1 && a.side[k].heads > 0) b = 1;  // writes dw even with no tokens
    a.side[k].blocks = (int32_t)b;
  }
}

template <typename E, int K, int H, bool HALF, bool BWD>
cudaError_t launch_vectors(NormArgs& a, cudaStream_t stream) {
  auto* kernel = norm_rope_kernel<E, K, H, HALF, BWD>;
  const int groups = kThreads / a.lanes, pairs = a.rope / 2;
  const size_t smem = sizeof(uint64_t) * ((pairs + 1) & ~1) + sizeof(float2) * pairs * groups;  // at most 20 KB
  const int64_t blocks = (int64_t)152 * occupancy((const void*)kernel, kThreads, smem);
  for (int k = 0; k < 2; ++k) {
    Side& s = a.side[k];
    // An item's heads share its sines: as many as leave each group of lanes two items.
    // (32768 tokens of 40 heads of 128, half turned: a batch an item 174 us, all heads 116.)
    s.span = H;
    while (s.span < s.heads && a.tokens * ((s.heads + 2 * s.span - 1) / (2 * s.span)) >= 2 * blocks * groups) s.span *= 2;
    s.groups = (s.heads + s.span - 1) / s.span;
    s.items = a.tokens * s.groups;
  }
  deal_out(a, groups, blocks);
  return launch_dependent(kernel, dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)), dim3(kThreads), smem, stream, a);
}

// One head a token, or several in flight.
template <typename E, int K, bool HALF, bool BWD>
cudaError_t launch_heads(NormArgs& a, cudaStream_t stream) {
  constexpr int columns = K * kChunk<E, HALF>, most = BWD ? 16 : 32;  // of a lane; in flight
  constexpr int H = columns < most ? most / columns : 1;
  if (a.side[0].heads == 1 && a.side[1].heads <= 1) return launch_vectors<E, K, 1, HALF, BWD>(a, stream);
  return launch_vectors<E, K, H, HALF, BWD>(a, stream);
}

template <typename E, bool HALF, bool BWD>
cudaError_t launch_kind(NormArgs& a, bool vectors, cudaStream_t stream) {
  constexpr int N = kChunk<E, HALF>;
  if (!vectors) {
    for (int k = 0; k < 2; ++k) a.side[k].items = a.tokens * a.side[k].heads;
    deal_out(a, kThreads / 32, 152 * 8);
    return launch_dependent(norm_rope_any_kernel<E, HALF, BWD>, dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)),
                            dim3(kThreads), 0, stream, a);
  }
  // units that lanes are dealt: vectors, or pairs of them; at most 128
  const int total = a.d / N, hp = a.rope / (2 * N);
  const int units = HALF ? hp + (total - 2 * hp + 1) / 2 : total;
  const int each = units <= 32 ? 1 : units <= 64 ? 2 : 4;
  a.lanes = 4;
  while (a.lanes < 32 && a.lanes * each < units) a.lanes *= 2;
  constexpr int V = HALF ? 2 : 1;  // vectors of a unit
  if (each == 1) return launch_heads<E, V, HALF, BWD>(a, stream);
  if (each == 2) return launch_heads<E, 2 * V, HALF, BWD>(a, stream);
  // fp32 in halves has at most 64 units: 128 vectors of 4 columns, two of them each
  if constexpr (!HALF || sizeof(E) == 2) return launch_heads<E, 4 * V, HALF, BWD>(a, stream);
  return cudaErrorInvalidValue;
}

template <typename E>
cudaError_t launch_norm(NormArgs& a, bool vectors, bool half, bool bwd, cudaStream_t stream) {
  if (!bwd) return half ? launch_kind<E, true, false>(a, vectors, stream) : launch_kind<E, false, false>(a, vectors, stream);
  const int64_t most = 152 * 32;  // CTAs: at most 16 of 128 threads an SM reside
  void* ws = nullptr;
  cudaError_t e = workspace_take(&ws, sizeof(float) * most * a.d, stream);
  if (e != cudaSuccess) return e;
  a.partial = static_cast<float*>(ws);
  e = half ? launch_kind<E, true, true>(a, vectors, stream) : launch_kind<E, false, true>(a, vectors, stream);
  if (e == cudaSuccess)
    e = launch_dependent(norm_weights_kernel<E>, dim3((unsigned)((a.d + 31) / 32), a.side[1].heads > 0 ? 2 : 1), dim3(32 * kLines), 0,
                         stream, a);
  const cudaError_t ef = workspace_give(ws, stream);
  return e != cudaSuccess ? e : ef;
}

// Strides of a tensor: no index may pass 63 bits.
bool strides_in_range(int64_t tokens, int32_t heads, int64_t ts, int64_t hs) {
  const int64_t most = (int64_t)1 << 60;
  return ts >= 0 && hs >= 0 && (tokens <= 1 || ts <= most / (tokens - 1)) && (heads <= 1 || hs <= most / (heads - 1));
}

// Heads within a token's stretch, or tokens within a head's.
bool distinct(int64_t tokens, int32_t heads, int32_t d, int64_t ts, int64_t hs) {
  if ((heads > 1 && hs < d) || (tokens > 1 && ts < d)) return false;
  return heads <= 1 || tokens <= 1 || ts >= (heads - 1) * hs + d || hs >= (tokens - 1) * ts + d;
}

csa_status_t call(const csa_norm_rope_t* how, const csa_norm_side_t* q, const csa_norm_side_t* k, bool bwd,
                  cudaStream_t stream) {
  if (!how || !q) return CSA_ERR_NULL;
  const csa_norm_rope_t& n = *how;
  if (n.dtype != CSA_BF16 && n.dtype != CSA_FP16 && n.dtype != CSA_FP32) return CSA_ERR_UNSUPPORTED;
  if (n.weight_dtype != n.dtype && n.weight_dtype != CSA_FP32) return CSA_ERR_UNSUPPORTED;
  if (n.layout != CSA_ROPE_INTERLEAVED && n.layout != CSA_ROPE_HALF) return CSA_ERR_UNSUPPORTED;
  if (n.rope_dim < 2 || n.rope_dim % 2 != 0 || n.offset < 0 || n.head_dim < 1 || n.head_dim > kMaxHeadDim ||
      (int64_t)n.offset + n.rope_dim > n.head_dim)
    return CSA_ERR_UNSUPPORTED;
  if (n.positions && n.position_bits != 32 && n.position_bits != 64) return CSA_ERR_UNSUPPORTED;
  if (n.tokens < 0 || !(n.eps >= 0.0f) || !isfinite(n.eps)) return CSA_ERR_RANGE;
  if (!n.freqs || (!n.positions && !n.cu_rows)) return CSA_ERR_NULL;
  if (!n.positions && (n.num_seqs < 1 || n.ratio < 1)) return CSA_ERR_RANGE;
  const uintptr_t size = n.dtype == CSA_FP32 ? 4 : 2, wsize = n.weight_dtype == CSA_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(n.freqs) % 8 != 0 || reinterpret_cast<uintptr_t>(n.cu_rows) % 4 != 0 ||
      (n.positions && reinterpret_cast<uintptr_t>(n.positions) % (n.position_bits / 8) != 0))
    return CSA_ERR_ALIGN;
  NormArgs a = {};
  const int vec = n.dtype == CSA_FP32 ? 4 : 8;
  // at most 128 vectors: 32 lanes of 4
  bool vectors = n.head_dim % vec == 0 && n.head_dim / vec <= 128 && n.offset % vec == 0 &&
                 n.rope_dim % (n.layout == CSA_ROPE_HALF ? 2 * vec : vec) == 0;
  for (int i = 0; i < 2; ++i) {
    const csa_norm_side_t* s = i ? k : q;
    if (!s) continue;
    if (s->heads < 1 || n.tokens > ((int64_t)1 << 60) / s->heads / n.head_dim) return CSA_ERR_RANGE;
    if (!strides_in_range(n.tokens, s->heads, s->x_token_stride, s->x_head_stride) ||
        !strides_in_range(n.tokens, s->heads, s->y_token_stride, s->y_head_stride) ||
        (bwd && !strides_in_range(n.tokens, s->heads, s->grad_token_stride, s->grad_head_stride)))
      return CSA_ERR_RANGE;
    if (!distinct(n.tokens, s->heads, n.head_dim, s->y_token_stride, s->y_head_stride)) return CSA_ERR_RANGE;
    if (!s->weight || (bwd && !s->dweight)) return CSA_ERR_NULL;
    if (n.tokens > 0 && (!s->x || !s->y || (bwd && !s->grad))) return CSA_ERR_NULL;
    const uintptr_t at = reinterpret_cast<uintptr_t>(s->x) | reinterpret_cast<uintptr_t>(s->y) |
                         (bwd ? reinterpret_cast<uintptr_t>(s->grad) : 0);
    const uintptr_t wat = reinterpret_cast<uintptr_t>(s->weight) | (bwd ? reinterpret_cast<uintptr_t>(s->dweight) : 0);
    if (at % size != 0 || wat % wsize != 0) return CSA_ERR_ALIGN;
    Side& t = a.side[i];
    // the stride of a single element is never stepped
    const bool many = n.tokens > 1, more = s->heads > 1;
    auto same = [&](const void* p, int64_t ts, int64_t hs) {
      return p != s->y || ((!many || ts == s->y_token_stride) && (!more || hs == s->y_head_stride));
    };
    if (n.tokens > 0 && (!same(s->x, s->x_token_stride, s->x_head_stride) ||
                         (bwd && !same(s->grad, s->grad_token_stride, s->grad_head_stride))))
      return CSA_ERR_RANGE;
    t.x = s->x;
    t.weight = s->weight;
    t.grad = s->grad;
    t.y = s->y;
    t.dweight = s->dweight;
    t.heads = s->heads;
    t.xt = many ? s->x_token_stride : 0;
    t.xh = more ? s->x_head_stride : 0;
    t.yt = many ? s->y_token_stride : 0;
    t.yh = more ? s->y_head_stride : 0;
    t.gt = many && bwd ? s->grad_token_stride : 0;
    t.gh = more && bwd ? s->grad_head_stride : 0;
    if (at % 16 != 0 || (t.xt | t.xh | t.yt | t.yh | t.gt | t.gh) % vec != 0) vectors = false;
  }
  if (n.tokens == 0 && !bwd) return CSA_OK;
  a.freqs = n.freqs;
  a.positions = n.positions;
  a.cu = n.cu_rows;
  a.tokens = n.tokens;
  a.position_bits = n.position_bits;
  a.nseq = n.num_seqs;
  a.ratio = n.ratio;
  for (int64_t step = 1; !n.positions && step < n.num_seqs; step *= 2) a.search = (int32_t)step;
  a.d = n.head_dim;
  a.rope = n.rope_dim;
  a.offset = n.offset;
  a.weight32 = n.weight_dtype == CSA_FP32;
  a.amplitude = n.amplitude;
  a.eps = n.eps;
  const bool half = n.layout == CSA_ROPE_HALF;
  const cudaError_t e = n.dtype == CSA_BF16   ? launch_norm<Bf16>(a, vectors, half, bwd, stream)
                        : n.dtype == CSA_FP16 ? launch_norm<__half>(a, vectors, half, bwd, stream)
                                              : launch_norm<float>(a, vectors, half, bwd, stream);
  return e == cudaSuccess ? CSA_OK : record_cuda_error(e);
}

}  // namespace

}  // namespace csa

extern "C" csa_status_t csa_norm_rope(const csa_norm_rope_t* how, const csa_norm_side_t* q,
                                      const csa_norm_side_t* k, cudaStream_t stream) {
  return csa::call(how, q, k, false, stream);
}

extern "C" csa_status_t csa_norm_rope_bwd(const csa_norm_rope_t* how, const csa_norm_side_t* q,
                                          const csa_norm_side_t* k, cudaStream_t stream) {
  return csa::call(how, q, k, true, stream);
}
