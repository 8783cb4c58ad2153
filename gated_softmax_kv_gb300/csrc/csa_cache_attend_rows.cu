// Attention over the 8-bit cache for tiles of 8 or 16 query rows (a decoding
// step's heads of one cache head; few tokens): memory-bound, mma.sync.
//
// Everything is computed transposed, so that the query rows are the N of the
// matrix instructions (8 a tile: a group of 8 heads wastes nothing):
//   S^T [16 keys x 8 rows] = K [16 x D] Q^T,  O^T [D x 8] += V^T [D x 16] P^T.
// A warp takes 16 or 32 keys a step on its own; heads of 256 and 512 columns
// are split over 2 and 4 warps, which add up their parts of S^T in shared
// memory. Keys arrive by cp.async in a ring of the warp's own; nothing but the
// end of an item makes the warps of a CTA wait for one another.
//
// The 8-bit values become fp16, which is exact. The order of a product's
// inner index is free, so a thread takes 16 consecutive columns of a key for
// four instructions, and V is transposed by byte permutes of the four keys
// that a thread's operand holds.
//
// Numerics. Queries are scaled row by row by a power of two into fp16, the row's
// largest value into [2^14, 2^15): exact for values down to 2^-31 of it (bf16) or
// 2^-28 (fp16), below that off by at most half a subnormal step, 2^-25, which is
// 2^-39 of it. The logits are fp32, in units of log2. With z_j the logit and s_j the value block's scale, the sum of weights
// is sum 2^(z_j - m) in fp32, and the weights of the second product are
// w_j = 2^(z_j + log2 s_j - m') in fp16: m' follows z + log2 s, so the scale is
// part of the weight and far apart scales cost no precision. Both references
// are raised only when a value passes them by 2^60 (m) or 2^8 (m'); w_j stays
// below 2^15, and what fp16 drops is below 2^-31 of the largest weight.
//
// Measured: 32 sequences of 5600 rows on average, 8 cache heads of 128 columns
// with 8 query heads each: 365 MB in 74 us (4.9 TB/s, 73% of the copy rate), the
// arithmetic units busy for 60% of it. One sequence of 300 rows of 512 columns
// by 16 heads: 13.9 us by a cluster of 8 blocks, 21.5 by one block.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache_attend.h"
#include "csa_cache_join.cuh"
#include "csa_cache_plan.cuh"
#include "csa_device.cuh"
#include "csa_e4m3.cuh"

namespace csa {

namespace {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ uint32_t smem_of(uint32_t at, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
template <bool CLUSTER>
__device__ __forceinline__ float4 load_shared(uint32_t at) {
  float4 v;
  if (CLUSTER)
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  else
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
constexpr int kMostSplit = 8;  // blocks of a cluster

template <int D, bool SHARED, int NT>
struct Shape {
  static constexpr int DW = D < 128 ? D : 128;  // columns of a warp
  static constexpr int WD = D / DW;             // warps of a group, which share their keys
  static constexpr int GROUPS = 8 / WD;
  static constexpr int ROWS = 8 * NT;
  static constexpr int SUB = SHARED && NT == 2 ? 2 : 1;  // 16-key parts of a step
  static constexpr int KS = 16 * SUB;
  static constexpr int PLANES = SHARED ? 1 : 2;
  static constexpr int TILE = 16 * DW;
  static constexpr int STAGE = SUB * (PLANES * TILE + 128);  // + 32 scales
  static constexpr int PER_SM = NT == 1 ? 2 : 1;
  static constexpr int STAGES = NT == 2 || SHARED ? 5 : 3;
  static constexpr int RING = STAGES * STAGE;   // of one warp
  static constexpr int XCHG = WD > 1 ? 2 * 8 * 32 * 4 * SUB * NT * 4 : 0;  // two buffers of S^T parts
  static constexpr int MERGE = GROUPS * ROWS * (D + 4) * 4;
  static constexpr int BODY = 8 * RING > MERGE ? 8 * RING : MERGE;  // the ring, Q and the merge in turn
  static constexpr int SMEM = BODY + XCHG;
  static_assert(ROWS * D * 2 <= BODY, "Q is staged where the ring will be");
  // A slot of the workspace: the rows' sums of D columns, then m, m', l.
  static constexpr int SLOT = ROWS * (D + 4);
};

// 16-byte chunk that chunk ch of key k lies in: conflict-free for both reads
// (K: 2 keys x 4 chunks a quarter warp, V: 4 keys x 2 chunks).
template <int DW>
__device__ __forceinline__ int swizzled(int k, int ch) {
  if constexpr (DW == 128)
    return ch ^ ((k & 6) ^ ((k & 1) << 2));
  else
    return ch ^ ((k >> 1) & 3);
}

// Where column c (a multiple of 4) of a row lies in a group's sums: the four
// rows that a quarter warp stores to are kept on different banks.
template <int DW>
__device__ __forceinline__ int merged_at(int row, int c) {
  const int t = (row >> 1) & 3;
  return c ^ ((DW == 128 ? t : (t & 1) | ((t & 2) << 1)) << 2);
}

template <int D, bool SHARED, int NT, bool HALF, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, CLUSTER ? 1 : Shape<D, SHARED, NT>::PER_SM)
    attend_rows_kernel(const AttendArgs a, const PlanShape plan) {
  using C = Shape<D, SHARED, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sums[kThreads / 32 + 1];
  __shared__ Place found;
  __shared__ int32_t row_sees[C::ROWS];
  __shared__ float row_factor[C::ROWS];
  __shared__ int64_t row_at[C::ROWS];                  // where its output row is, or -1
  __shared__ float merged[C::ROWS], part_factor[(CLUSTER ? kMostSplit : 1) * C::GROUPS][C::ROWS];
  __shared__ int32_t sees_least, sees_most;
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int grp = warp / C::WD, wd = warp % C::WD;
  uint8_t* ring = smem + warp * C::RING;
  const uint32_t ring_at = smem_addr(ring);
  const int split = CLUSTER ? plan.split : 1, rank = CLUSTER ? blockIdx.x & (split - 1) : 0;
  const int stride = C::GROUPS * split;  // chunks of a step of the worker
  const Place place = locate<kThreads>(a, plan, CLUSTER ? blockIdx.x / split : blockIdx.x, sums, &found);
  Shared* left = shared_items<C::ROWS, D>(a, plan.workers) + blockIdx.x;  // unless items are whole
  if (place.pos < 0) {
    if (threadIdx.x == 0 && !plan.whole) left->parts = 0;
    return;
  }
  Shared tail = {0, 0, 0, 0};  // an item that begins here and ends with another worker
  const int pb = a.c.page_bits, bb = a.c.block_bits;

  int s = place.s;
  SeqWork work = seq_work(a, plan, s);
  int64_t within = place.within;
  for (int64_t pos = place.pos; pos < place.end;) {
    if (within >= work.tiles * work.chunks * a.kv) {  // the next sequence with queries
      ++s;
      work = seq_work(a, plan, s);
      within = 0;
      continue;
    }
    const int64_t item = within / work.chunks;
    const int64_t c0 = within - item * work.chunks;
    const int h = (int)(item / work.tiles);
    const int64_t tile = item - h * work.tiles;
    const int64_t units = plan.whole ? 1 : min(work.chunks - c0, place.end - pos);
    const int64_t c1 = plan.whole ? (int64_t)1 << 40 : c0 + units;
    const bool whole = plan.whole || units == work.chunks;
    if (c0 == 0 && !whole)
      tail = {1 + (int32_t)((work.chunks - c1 + place.per - 1) / place.per), s, (int32_t)tile, h};

    // ---- the rows: what they see, and Q as fp16 --------------------------------
    __syncthreads();  // the last item is out of shared memory
    if (threadIdx.x == 0) {
      sees_least = 0x7FFFFFFF;
      sees_most = 0;
    }
    __syncthreads();
    uint16_t* qs = reinterpret_cast<uint16_t*>(smem);
    constexpr int V = D / 256 > 0 ? D / 256 : 1;  // 16-byte vectors a lane
    Row rows[NT];
    uint4 x[NT][V];
#pragma unroll
    for (int r = 0; r < NT; ++r) {  // all loads first
      rows[r] = row_of(a, s, tile, h, C::ROWS, warp + 8 * r);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int col = (k * 32 + lane) * 8;
        x[r][k] = rows[r].there && col < D ? __ldg(reinterpret_cast<const uint4*>(
                                                 a.q + rows[r].token * a.qt + rows[r].head * a.qh + col))
                                           : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int i = warp + 8 * r;
      const Row& w = rows[r];
      if (lane == 0) {
        int64_t n = w.there ? work.keys : 0;
        if (w.there && a.visible) n = min(n, (int64_t)max(__ldg(a.visible + w.token), 0));
        row_sees[i] = w.there ? (int)n : -1;
        row_at[i] = w.there ? w.token * a.heads + w.head : -1;
        if (w.there) {
          atomicMin(&sees_least, (int)n);
          atomicMax(&sees_most, (int)n);
        }
      }
      const int lift = query_lift<HALF>(finite_max<HALF, V>(x[r]));
      const float f = exp2i(lift);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int col = (k * 32 + lane) * 8;
        if (col < D) *reinterpret_cast<uint4*>(qs + i * D + col) = lifted<HALF>(x[r][k], f);
      }
      if (lane == 0) row_factor[i] = a.scale * exp2i(-lift);
    }
    __syncthreads();
    uint32_t qf[NT][C::DW / 16][2];
    float zf[NT][2];
    int sees[NT][2];
    const int least = sees_least, most = sees_most;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < C::DW / 16; ++k) {
        const uint2 x = *reinterpret_cast<const uint2*>(
            qs + (n * 8 + g) * D + wd * C::DW + (k >> 2) * 64 + 16 * t + 4 * (k & 3));
        qf[n][k][0] = x.x;
        qf[n][k][1] = x.y;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        zf[n][j] = row_factor[n * 8 + 2 * t + j];
        const int v = row_sees[n * 8 + 2 * t + j];
        sees[n][j] = v < 0 ? 0x7FFFFFFF : v;  // rows that are not there are not looked at
      }
    }
    __syncthreads();  // the ring takes Q's place

    // ---- the keys --------------------------------------------------------------
    const int64_t stop = min(c1, ((int64_t)most + C::KS - 1) / C::KS);
    const int64_t begin = c0 + rank * C::GROUPS + grp;
    const int steps = stop > begin ? (int)((stop - begin + stride - 1) / stride) : 0;
    const int32_t* row_table = a.table + (int64_t)s * a.max_pages;
    auto page_at = [&](int i, int u) -> int32_t {  // page of part u of step i
      if (i >= steps) return -1;
      const int64_t key = (begin + (int64_t)i * stride) * C::KS + u * 16;
      return key < most ? __ldg(row_table + (key >> pb)) : -1;
    };
    auto fetch = [&](int i, const int32_t* pages) {
      if (i < steps) {
        const uint32_t at = ring_at + (i % C::STAGES) * C::STAGE;
#pragma unroll
        for (int u = 0; u < C::SUB; ++u) {
          const int64_t key0 = (begin + (int64_t)i * stride) * C::KS + u * 16;
          const bool in = pages[u] >= 0 && pages[u] < a.c.num_pages && key0 < most;
          const int slot = (int)(key0 & ((1 << pb) - 1));
          const int left = (int)min((int64_t)16, most - key0);  // rows that some query sees
#pragma unroll
          for (int pl = 0; pl < C::PLANES; ++pl) {
            const int64_t chunk = (int64_t)(in ? pages[u] : 0) * a.c.heads + (pl ? a.v_first : 0) + h;
            const uint8_t* src = a.c.data + ((chunk << pb) + slot) * D + wd * C::DW;
            constexpr int PER = C::DW / 16;
#pragma unroll
            for (int k = 0; k < C::DW / 32; ++k) {
              const int unit = lane + 32 * k, key = unit / PER, ch = unit % PER;
              const bool ok = in && key < left;
              cp16(at + (u * C::PLANES + pl) * C::TILE + key * C::DW + (swizzled<C::DW>(key, ch) << 4),
                   ok ? src + key * D + ch * 16 : a.c.data, ok);
            }
          }
          // scales of the 16 keys, then of the 16 values; -1 where there is no row
          const int key = lane & 15;
          const uint32_t sc = at + C::SUB * C::PLANES * C::TILE + u * 128 + lane * 4;
          if (in && key < left) {
            const int64_t chunk = (int64_t)pages[u] * a.c.heads + (lane < 16 ? 0 : a.v_first) + h;
            cp4(sc, a.c.scales + (chunk << (pb - bb)) + ((slot + key) >> bb));
          } else {
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc), "f"(-1.0f) : "memory");
          }
        }
      }
      cp_commit();
    };

    float o[C::DW / 16][NT][4], m[NT][2], mp[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < C::DW / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[n][j] = mp[n][j] = kNone;
        l[n][j] = 0.0f;
      }
    // the first steps' lookups at once, a lane each
    const int32_t lookup = lane < C::STAGES * C::SUB ? page_at(lane / C::SUB, lane % C::SUB) : -1;
    int32_t pages[C::SUB];
#pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) {
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) pages[u] = __shfl_sync(0xFFFFFFFFu, lookup, i * C::SUB + u);
      if (i < C::STAGES - 1) fetch(i, pages);
    }

    for (int i = 0; i < steps; ++i) {
      cp_wait<C::STAGES - 2>();
      __syncwarp();  // the step has arrived, and the one before it is used up
      fetch(i + C::STAGES - 1, pages);
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) pages[u] = page_at(i + C::STAGES, u);
      const uint8_t* stage = ring + (i % C::STAGES) * C::STAGE;
      const float* scales = reinterpret_cast<const float*>(stage + C::SUB * C::PLANES * C::TILE);
      const int64_t key0 = (begin + (int64_t)i * stride) * C::KS;

      // S^T
      float sc[C::SUB][NT][4];
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[u][n][e] = 0.0f;
        const uint8_t* kt = stage + u * C::PLANES * C::TILE;
#pragma unroll
        for (int b = 0; b < C::DW / 64; ++b) {
          const uint4 x = *reinterpret_cast<const uint4*>(
              kt + g * C::DW + (swizzled<C::DW>(g, 4 * b + t) << 4));
          const uint4 y = *reinterpret_cast<const uint4*>(
              kt + (g + 8) * C::DW + (swizzled<C::DW>(g + 8, 4 * b + t) << 4));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = lo_f16x2(xs[j]), a1 = lo_f16x2(ys[j]);
            const uint32_t a2 = hi_f16x2(xs[j]), a3 = hi_f16x2(ys[j]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(sc[u][n], a0, a1, a2, a3, qf[n][4 * b + j][0], qf[n][4 * b + j][1]);
          }
        }
      }
      if constexpr (C::WD > 1) {  // the other columns' parts, added in the warps' order
        constexpr int N4 = C::SUB * NT;
        float4* buf = reinterpret_cast<float4*>(smem + C::BODY) + ((i & 1) * 8 + grp * C::WD) * 32 * N4;
#pragma unroll
        for (int u = 0; u < C::SUB; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            buf[(wd * N4 + u * NT + n) * 32 + lane] =
                make_float4(sc[u][n][0], sc[u][n][1], sc[u][n][2], sc[u][n][3]);
        group_barrier(1 + grp, 32 * C::WD);
#pragma unroll
        for (int u = 0; u < C::SUB; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float4 x = buf[(u * NT + n) * 32 + lane];
#pragma unroll
            for (int w = 1; w < C::WD; ++w) {
              const float4 y = buf[(w * N4 + u * NT + n) * 32 + lane];
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            sc[u][n][0] = x.x;
            sc[u][n][1] = x.y;
            sc[u][n][2] = x.z;
            sc[u][n][3] = x.w;
          }
      }

      // logits, their values with the scale (zp), and whether a reference is passed
      float zp[C::SUB][NT][4];
      bool masked = key0 + C::KS > least, up = false;
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) {
        const float k0 = scales[u * 32 + g], k1 = scales[u * 32 + g + 8];
        const float v0 = SHARED ? k0 : scales[u * 32 + 16 + g];
        const float v1 = SHARED ? k1 : scales[u * 32 + 24 + g];
        const bool gone0 = k0 < 0.0f, gone1 = k1 < 0.0f;
        masked = masked || __any_sync(0xFFFFFFFFu, gone0 || gone1);
        const float lv0 = __log2f(v0), lv1 = __log2f(v1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][n][e] *= (e < 2 ? k0 : k1) * zf[n][e & 1];
        if (masked) {
          const int64_t j0 = key0 + u * 16 + g;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((e < 2 ? gone0 : gone1) || (e < 2 ? j0 : j0 + 8) >= sees[n][e & 1])
                sc[u][n][e] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            zp[u][n][e] = sc[u][n][e] == -INFINITY ? -INFINITY : sc[u][n][e] + (e < 2 ? lv0 : lv1);
            up = up || sc[u][n][e] > m[n][e & 1] + kSlackM || zp[u][n][e] > mp[n][e & 1] + kSlackW;
          }
      }
      if (__any_sync(0xFFFFFFFFu, up)) {  // raise the references to the step's maxima
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = m[n][j], y = mp[n][j];
#pragma unroll
            for (int u = 0; u < C::SUB; ++u) {
              x = fmaxf(x, fmaxf(sc[u][n][j], sc[u][n][j + 2]));
              y = fmaxf(y, fmaxf(zp[u][n][j], zp[u][n][j + 2]));
            }
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, w));
            }
            l[n][j] *= ex2_approx_ftz(m[n][j] - x);
            const float f = ex2_approx_ftz(mp[n][j] - y);
#pragma unroll
            for (int k = 0; k < C::DW / 16; ++k) {
              o[k][n][j] *= f;
              o[k][n][j + 2] *= f;
            }
            m[n][j] = x;
            mp[n][j] = y;
          }
      }
      // weights
      uint32_t pf[C::SUB][NT][2];
#pragma unroll
      for (int u = 0; u < C::SUB; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[n][e & 1] += ex2_approx_ftz(sc[u][n][e] - m[n][e & 1]);
            w[e] = ex2_approx_ftz(zp[u][n][e] - (mp[n][e & 1] - kLift));
          }
          pf[u][n][0] = transpose8x8(pack_f16x2(w[0], w[1]));
          pf[u][n][1] = transpose8x8(pack_f16x2(w[2], w[3]));
        }

      // O^T
#pragma unroll
      for (int u = 0; u < C::SUB; ++u) {
        const uint8_t* vt = stage + (u * C::PLANES + C::PLANES - 1) * C::TILE;
        constexpr int W = C::DW / 32;  // words a key: 4 or 2
        uint32_t x[4][W];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 2 * t + (k & 1) + 8 * (k >> 1);
          if constexpr (W == 4) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(
                vt + key * C::DW + (swizzled<C::DW>(key, g) << 4));
            x[k][0] = q4.x;
            x[k][1] = q4.y;
            x[k][2] = q4.z;
            x[k][3] = q4.w;
          } else {
            const uint2 q2 = *reinterpret_cast<const uint2*>(
                vt + key * C::DW + (swizzled<C::DW>(key, g >> 1) << 4) + 8 * (g & 1));
            x[k][0] = q2.x;
            x[k][1] = q2.y;
          }
        }
        bool poison = false;
        if (masked) {  // a row that some queries do not see may hold NaN: 0 * NaN must not reach them
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < W; ++w) any |= nan_bytes(x[k][w]);
          poison = __any_sync(0xFFFFFFFFu, any != 0);
        }
        if (poison) {
          // Counts, for each (column, row), the NaN that the row does see, and
          // takes the NaN out of the product itself.
          uint32_t seen[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = sc[u][n][e] == -INFINITY ? 0.0f : 1.0f;
            seen[n][0] = transpose8x8(pack_f16x2(v[0], v[1]));
            seen[n][1] = transpose8x8(pack_f16x2(v[2], v[3]));
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t bad = nan_bytes(x[k][w]);
              b[k] = bad & 0x38383838u;  // 1.0
              x[k][w] &= ~bad;
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t lo = __byte_perm(b[0], b[1], hf ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(b[2], b[3], hf ? 0x7362 : 0x5140);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16816(c, lo_f16x2(lo), hi_f16x2(lo), lo_f16x2(hi), hi_f16x2(hi), seen[n][0], seen[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (c[e] > 0.0f) o[2 * w + hf][n][e] = NAN;
              }
            }
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t lo = __byte_perm(x[0][w], x[1][w], hf ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(x[2][w], x[3][w], hf ? 0x7362 : 0x5140);
            const uint32_t a0 = lo_f16x2(lo), a1 = hi_f16x2(lo), a2 = lo_f16x2(hi), a3 = hi_f16x2(hi);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(o[2 * w + hf][n], a0, a1, a2, a3, pf[u][n][0], pf[u][n][1]);
          }
      }
    }
    cp_wait<0>();
    __syncthreads();  // the merge takes the ring's place

    // ---- the groups' results, then the item's ------------------------------------
    float* mg = reinterpret_cast<float*>(smem) + grp * C::SLOT;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = n * 8 + 2 * t + j;
        float x = l[n][j];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
        if (wd == 0 && g == 0) {
          mg[C::ROWS * D + row * 4] = m[n][j];
          mg[C::ROWS * D + row * 4 + 1] = mp[n][j];
          mg[C::ROWS * D + row * 4 + 2] = x;
        }
#pragma unroll
        for (int k = 0; k < C::DW / 16; k += 2)
          *reinterpret_cast<float4*>(mg + row * D + merged_at<C::DW>(row, wd * C::DW + g * (C::DW / 8) + 2 * k)) =
              make_float4(o[k][n][j], o[k][n][j + 2], o[k + 1][n][j], o[k + 1][n][j + 2]);
      }
    if constexpr (CLUSTER)
      cluster_barrier();
    else
      __syncthreads();
    // A warp a row: its statistics over the groups (a lane each), and the factor
    // of each group's sums, with which they are finished or (split items) joined.
    // The blocks of a cluster share the rows out.
    const uint32_t parts = smem_addr(smem);
    const int n = stride, own = C::ROWS / split, row0 = rank * own;
    auto part_at = [&](int k) -> uint32_t {  // of group k of the worker
      if (!CLUSTER) return parts + k * (C::SLOT * 4);
      return smem_of(parts + (k % C::GROUPS) * (C::SLOT * 4), k / C::GROUPS);
    };
    // slot 0: the item began with another worker, slot 1: it did here
    float* const ws = a.ws + ((int64_t)blockIdx.x * 2 + (c0 == 0)) * C::SLOT;
    for (int row = row0 + warp; row < row0 + own; row += 8) {
      constexpr int LANES = CLUSTER ? kMostSplit * C::GROUPS / 32 + (kMostSplit * C::GROUPS < 32) : 1;
      float4 st[LANES];
      RowStats r = {kNone, kNone, 0.0f};
#pragma unroll
      for (int k = 0; k < LANES; ++k) {
        st[k] = make_float4(kNone, kNone, 0.0f, 0.0f);
        if (lane + 32 * k < n) st[k] = load_shared<CLUSTER>(part_at(lane + 32 * k) + (C::ROWS * D + row * 4) * 4);
        r.m = fmaxf(r.m, st[k].x);
        r.mp = fmaxf(r.mp, st[k].y);
      }
#pragma unroll
      for (int w = 16; w; w >>= 1) {
        r.m = fmaxf(r.m, __shfl_xor_sync(0xFFFFFFFFu, r.m, w));
        r.mp = fmaxf(r.mp, __shfl_xor_sync(0xFFFFFFFFu, r.mp, w));
      }
#pragma unroll
      for (int k = 0; k < LANES; ++k) r.l += st[k].z * exp2f(st[k].x - r.m);
#pragma unroll
      for (int w = 16; w; w >>= 1) r.l += __shfl_xor_sync(0xFFFFFFFFu, r.l, w);
      const float up = whole ? r.m + kLift + log2f(r.l) : r.mp;
#pragma unroll
      for (int k = 0; k < LANES; ++k)
        if (lane + 32 * k < n) part_factor[lane + 32 * k][row] = exp2f(st[k].y - up);
      if (lane == 0) {
        merged[row] = r.l;
        if (!whole)
          *reinterpret_cast<float4*>(ws + C::ROWS * D + row * 4) = make_float4(r.m, r.mp, r.l, 0.0f);
        else if (a.lse && row_at[row] >= 0)
          a.lse[row_at[row]] = row_lse(r);
      }
    }
    __syncthreads();
#pragma unroll 2
    for (int u = threadIdx.x; u < own * (D / 4); u += kThreads) {
      const int row = row0 + u / (D / 4), c = (u % (D / 4)) * 4;
      const uint32_t at = (row * D + merged_at<C::DW>(row, c)) * 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int b = 0; b < split; ++b) {
        const uint32_t from = part_at(b * C::GROUPS) + at;
#pragma unroll
        for (int k = 0; k < C::GROUPS; ++k) {
          const float4 x = load_shared<CLUSTER>(from + k * (C::SLOT * 4));
          const float f = part_factor[b * C::GROUPS + k][row];
          v.x = fmaf(x.x, f, v.x);
          v.y = fmaf(x.y, f, v.y);
          v.z = fmaf(x.z, f, v.z);
          v.w = fmaf(x.w, f, v.w);
        }
      }
      if (!whole)
        *reinterpret_cast<float4*>(ws + row * D + c) = v;
      else if (row_at[row] >= 0)
        store4<HALF>(a.out + row_at[row] * D + c, v, merged[row] == 0.0f ? 0.0f : 1.0f);
    }
    if (CLUSTER) cluster_barrier();  // the other blocks have read this one's sums
    pos += units;
    within += units;
  }
  if (threadIdx.x == 0 && !plan.whole) *left = tail;
}

template <int D, bool SHARED, int NT, bool HALF>
cudaError_t launch_tile(AttendArgs a, cudaStream_t stream) {
  using C = Shape<D, SHARED, NT>;
  const PlanShape p = plan_of(a, C::ROWS, C::KS, 152 * C::PER_SM, 2 * C::GROUPS, 8 * C::GROUPS, C::GROUPS);
  if (p.split > 1) {
    auto* kernel = attend_rows_kernel<D, SHARED, NT, HALF, true>;
    const cudaError_t e = allow_dynamic_smem((const void*)kernel, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_clusters(kernel, dim3((unsigned)(p.workers * p.split)), dim3(kThreads), C::SMEM, (unsigned)p.split,
                           stream, a, p);
  }
  auto* kernel = attend_rows_kernel<D, SHARED, NT, HALF, false>;
  cudaError_t e = allow_dynamic_smem((const void*)kernel, C::SMEM);
  if (e != cudaSuccess) return e;
  if (p.whole)
    return launch_dependent(kernel, dim3((unsigned)p.workers), dim3(kThreads), C::SMEM, stream, a, p);
  void* ws = nullptr;
  e = workspace_take(&ws, join_bytes<D, C::ROWS>(p.workers), stream);
  if (e != cudaSuccess) return e;
  a.ws = static_cast<float*>(ws);
  e = launch_dependent(kernel, dim3((unsigned)p.workers), dim3(kThreads), C::SMEM, stream, a, p);
  if (e == cudaSuccess) e = launch_join<D, C::ROWS, HALF>(a, p.workers, stream);
  const cudaError_t ef = workspace_give(ws, stream);
  return e != cudaSuccess ? e : ef;
}

template <int D, bool SHARED, bool HALF>
cudaError_t launch_rows(const AttendArgs& a, cudaStream_t stream) {
  // A tile of 8 rows holds a group of up to 8 heads; larger groups, and more
  // than one token a sequence, fill 16 rows for one pass over the keys. Measured
  // (32 sequences, tiles of 8 against 16): 8 cache heads of 128 with 8 heads each
  // 78 us / 122, with 16 each 141 / 123; one of 512 with 8 heads 29 / 34, with 16
  // heads 43 / 35.
  if (a.group <= 8 && (int64_t)a.group * a.tokens <= (int64_t)8 * a.nseq)
    return launch_tile<D, SHARED, 1, HALF>(a, stream);
  return launch_tile<D, SHARED, 2, HALF>(a, stream);
}

template <int D>
cudaError_t launch_dim(const AttendArgs& a, bool half, bool shared, cudaStream_t stream) {
  if (shared)
    return half ? launch_rows<D, true, true>(a, stream) : launch_rows<D, true, false>(a, stream);
  return half ? launch_rows<D, false, true>(a, stream) : launch_rows<D, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_attend_rows(const AttendArgs& a, bool half, bool shared, cudaStream_t stream) {
  switch (a.c.d) {
    case 64: return launch_dim<64>(a, half, shared, stream);
    case 128: return launch_dim<128>(a, half, shared, stream);
    case 256: return launch_dim<256>(a, half, shared, stream);
    default: return launch_dim<512>(a, half, shared, stream);
  }
}

}  // namespace csa
