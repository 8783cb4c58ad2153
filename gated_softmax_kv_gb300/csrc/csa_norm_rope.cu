// Norms of queries and keys for each head with the rotary positions in the same
// pass, and their gradient (declared in include/csa_norm_rope.h).
//
// A group of G lanes (4 .. 32) owns a head: a lane holds K vectors of 16 bytes of
// it, so a mean over the head is log2(G) shuffles and each byte is read once. For
// the half layout a lane's vectors come in pairs half a part apart, so that both
// columns of a pair are its own. A group keeps its columns for its whole loop:
// frequencies and weights are worked out once, and the sines of a token serve
// HEADS heads of it, whose loads are issued before the sines are worked out.
//
// The gradient reads x and grad once, works r out again, and sums its part of dw
// in registers over the loop; the groups' sums meet in shared memory in a fixed
// order, and a second kernel adds the CTAs' in theirs.
//
// Angles are those of csa_rope.cu. Memory bounds both directions.
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
  int32_t groups;  // of heads, a token
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

template <typename E>
__device__ __forceinline__ float weight_at(const NormArgs& a, const Side& s, int c) {
  return a.weight32 ? __ldg(static_cast<const float*>(s.weight) + c) : Elem<E>::load(static_cast<const E*>(s.weight) + c);
}

// Sum over the G lanes of a group (a power of two), the same in each.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
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

// The turn of a group's vectors, and its transpose (sn negated): vectors 2j and
// 2j + 1 are the two halves of the same pairs, or a vector has whole pairs.
template <int N, int K, bool HALF>
__device__ __forceinline__ void turn_vectors(float (&v)[K][N], const int (&pair)[K], const float (&cs)[K][N / 2],
                                             const float (&sn)[K][N / 2], float sign) {
  if constexpr (HALF) {
#pragma unroll
    for (int k = 0; k < K; k += 2)
      if (pair[k] >= 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float c = cs[k + i / (N / 2)][i % (N / 2)], s = sign * sn[k + i / (N / 2)][i % (N / 2)];
          const float x = v[k][i], y = v[k + 1][i];
          v[k][i] = fmaf(-y, s, x * c);
          v[k + 1][i] = fmaf(x, s, y * c);
        }
      }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (pair[k] >= 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float c = cs[k][i], s = sign * sn[k][i];
          const float x = v[k][2 * i], y = v[k][2 * i + 1];
          v[k][2 * i] = fmaf(-y, s, x * c);
          v[k][2 * i + 1] = fmaf(x, s, y * c);
        }
      }
  }
}

template <typename E, int K, bool HALF, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<E>::N;
  constexpr int H = BWD ? 2 : K >= 4 ? 2 : 4;  // heads of an item
  __shared__ float sums[BWD ? kMaxHeadDim : 1];
  grid_dependency_wait();
  allow_dependent_launch();
  const bool second = (int)blockIdx.x >= a.side[0].blocks;
  const Side& s = a.side[second];
  const int block = (int)blockIdx.x - (second ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & (a.lanes - 1), group = threadIdx.x / a.lanes, groups = kThreads / a.lanes;
  int col[K], pair[K];
  columns_of<N, K, HALF>(a, lane, col, pair);
  uint64_t f[K][N / 2];
  float w[K][N];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      f[k][i] = pair[k] >= 0 ? turns_of(__ldg(a.freqs + pair[k] + (HALF ? (k & 1) * (N / 2) : 0) + i)) : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) w[k][i] = col[k] >= 0 ? weight_at<E>(a, s, col[k] + i) : 0.0f;
  }
  float dw[BWD ? K : 1][N];
#pragma unroll
  for (int k = 0; k < (BWD ? K : 1); ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[k][i] = 0.0f;
  const float inv_d = 1.0f / (float)a.d;
  const int64_t step = (int64_t)s.blocks * groups;
  // every group of a warp makes the same number of rounds: shuffles need all lanes
  const int64_t rounds = (s.items + step - 1) / step;
  for (int64_t n = 0; n < rounds; ++n) {
    const int64_t it = n * step + (int64_t)block * groups + group;
    const bool on = it < s.items;
    const int64_t token = on ? it / s.groups : 0;
    const int head = on ? (int)(it - token * s.groups) * H : 0;
    const int heads = on ? min(H, s.heads - head) : 0;
    uint4 xr[H][K], gr[BWD ? H : 1][K];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool there = h < heads && col[k] >= 0;
        xr[h][k] = there ? *reinterpret_cast<const uint4*>(static_cast<const E*>(s.x) + token * s.xt + (head + h) * s.xh + col[k])
                         : make_uint4(0, 0, 0, 0);
        if constexpr (BWD)
          gr[h][k] = there ? *reinterpret_cast<const uint4*>(static_cast<const E*>(s.grad) + token * s.gt + (head + h) * s.gh + col[k])
                           : make_uint4(0, 0, 0, 0);
      }
    float cs[K][N / 2], sn[K][N / 2];
    const int64_t pos = on ? position_of(a, token) : 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (pair[k] >= 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) turn_of(f[k][i], pos, a.amplitude, 1.0f, &cs[k][i], &sn[k][i]);
      }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float x[K][N], sum = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Vec<E>::unpack(xr[h][k], x[k]);
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(x[k][i], x[k][i], sum);
      }
      const float r = 1.0f / sqrtf(fmaf(group_sum(sum, a.lanes), inv_d, a.eps));
      if constexpr (!BWD) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < N; ++i) x[k][i] = x[k][i] * r * w[k][i];
        turn_vectors<N, K, HALF>(x, pair, cs, sn, 1.0f);
      } else {
        float g[K][N], along = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) Vec<E>::unpack(gr[h][k], g[k]);
        turn_vectors<N, K, HALF>(g, pair, cs, sn, -1.0f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (h < heads) dw[k][i] = fmaf(g[k][i], x[k][i] * r, dw[k][i]);
            g[k][i] *= w[k][i];
            along = fmaf(g[k][i], x[k][i], along);
          }
        const float back = group_sum(along, a.lanes) * inv_d * r * r;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < N; ++i) x[k][i] = r * fmaf(-x[k][i], back, g[k][i]);
      }
      if (h < heads) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (col[k] >= 0)
            *reinterpret_cast<uint4*>(static_cast<E*>(s.y) + token * s.yt + (head + h) * s.yh + col[k]) = Vec<E>::pack(x[k]);
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
            for (int i = 0; i < N; ++i) sums[col[k] + i] = turn == 0 ? dw[k][i] : sums[col[k] + i] + dw[k][i];
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

// dw of both sides from the CTAs' sums: 32 columns a CTA, 8 lines of CTAs summed
// apart and then in order.
template <typename E>
__global__ void __launch_bounds__(256) norm_weights_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[8][32];
  grid_dependency_wait();
  allow_dependent_launch();
  const Side& s = a.side[blockIdx.y];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), line = threadIdx.x >> 5;
  const float* p = a.partial + (int64_t)(blockIdx.y ? a.side[0].blocks : 0) * a.d;
  float v = 0.0f;
  if (c < a.d) {
#pragma unroll 8
    for (int b = line; b < s.blocks; b += 8) v += p[(int64_t)b * a.d + c];
  }
  part[line][threadIdx.x & 31] = v;
  __syncthreads();
  if (line == 0 && c < a.d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += part[k][threadIdx.x];
    if (a.weight32)
      static_cast<float*>(s.dweight)[c] = v;
    else
      Elem<E>::store(static_cast<E*>(s.dweight) + c, v);
  }
}

// CTAs of the two sides: as many as there is work for, at most `most` together,
// shared in proportion to their items.
void deal_out(NormArgs& a, int64_t per_block, int64_t most) {
  int64_t want[2];
  for (int k = 0; k < 2; ++k) want[k] = (a.side[k].items + per_block - 1) / per_block;
  const int64_t all = want[0] + want[1];
  for (int k = 0; k < 2; ++k) {
    int64_t b = all > most ? want[k] * most / all : want[k];
    if (b < 1 && a.side[k].heads > 0) b = 1;  // writes dw even with no tokens
    a.side[k].blocks = (int32_t)b;
  }
}

template <typename E, int K, bool HALF, bool BWD>
cudaError_t launch_vectors(NormArgs& a, cudaStream_t stream) {
  constexpr int H = BWD ? 2 : K >= 4 ? 2 : 4;
  for (int k = 0; k < 2; ++k) {
    a.side[k].groups = (a.side[k].heads + H - 1) / H;
    a.side[k].items = a.tokens * a.side[k].groups;
  }
  auto* kernel = norm_rope_kernel<E, K, HALF, BWD>;
  deal_out(a, kThreads / a.lanes, (int64_t)152 * occupancy((const void*)kernel, kThreads, 0));
  return launch_dependent(kernel, dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)), dim3(kThreads), 0, stream, a);
}

template <typename E, bool HALF, bool BWD>
cudaError_t launch_kind(NormArgs& a, bool vectors, cudaStream_t stream) {
  constexpr int N = Vec<E>::N;
  if (!vectors) {
    for (int k = 0; k < 2; ++k) a.side[k].items = a.tokens * a.side[k].heads;
    deal_out(a, kThreads / 32, 152 * 8);
    return launch_dependent(norm_rope_any_kernel<E, HALF, BWD>, dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)),
                            dim3(kThreads), 0, stream, a);
  }
  // units that lanes are dealt: vectors, or pairs of them
  const int total = a.d / N, hp = a.rope / (2 * N);
  const int units = HALF ? hp + (total - 2 * hp + 1) / 2 : total;
  auto lanes_for = [&](int each) {
    int n = 4;
    while (n < 32 && n * each < units) n *= 2;
    return n;
  };
  if (HALF) {
    const int each = units <= 32 ? 1 : 2;
    a.lanes = lanes_for(each);
    return each == 1 ? launch_vectors<E, 2, HALF, BWD>(a, stream) : launch_vectors<E, 4, HALF, BWD>(a, stream);
  }
  const int each = units <= 32 ? 1 : units <= 64 ? 2 : 4;
  a.lanes = lanes_for(each);
  if constexpr (!HALF) {
    if (each == 1) return launch_vectors<E, 1, HALF, BWD>(a, stream);
    if (each == 2) return launch_vectors<E, 2, HALF, BWD>(a, stream);
  }
  return launch_vectors<E, 4, HALF, BWD>(a, stream);
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
    e = launch_dependent(norm_weights_kernel<E>, dim3((unsigned)((a.d + 31) / 32), a.side[1].heads > 0 ? 2 : 1), dim3(256), 0,
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
