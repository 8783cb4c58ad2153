// Causal attention over packed sequences, forward: tcgen05.
//
// A CTA has two tiles of 128 query rows (csa_prompt_tile.cuh) and runs over the keys
// 128 at a time. For each tile
//   S [128 rows x 128 keys] = Q K^T           (TMEM, 128 columns)
//   O [128 rows x D] += P V                   (TMEM; P in S's place, two weights a column)
// with the running maximum and sum of a softmax, a row a thread. While one tile's
// softmax is under way the other's products are: the matrix instructions of a block,
// PV of tile t and then its next Q K^T, take as long as the softmax of the other.
//
// Roles: four warps a tile for its softmax and its result, one warp for the matrix
// instructions, one for TMA. Tiles of K and V come in a ring, in the order in which
// the instructions use them. Where only one tile has rows (single tokens, short
// prompts) both softmax groups work on it, on alternate blocks of keys, and add up
// at the end.
//
// The reference that logits are taken from rises only when they pass it by 2^8, so
// that O is seldom scaled: weights are at most 2^8. fp16 weights are lifted by
// another 2^7, so that small ones keep their bits; the factor cancels. Sums of
// weights are of what is not rounded yet.
//
// Blocks that some row of the CTA does not see in full are cleaned of infinities and
// NaN in V, which a weight of 0 would not keep out; rows that do see one get it back
// from memory at the end.
//
// Every wait on an mbarrier is bounded: a wait that runs out marks the CTA, whose
// later waits return at once and whose results become NaN.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "csa_internal.h"
#include "csa_prompt_tile.cuh"

namespace csa {

namespace {

template <int DP_, bool HALF_>
struct Fwd {
  static constexpr int DP = DP_;                  // columns, padded to a slab of 64
  static constexpr bool HALF = HALF_;
  static constexpr int SLAB = 16384;              // 128 rows x 64 columns
  static constexpr int TILE = DP / 64 * SLAB;
  static constexpr int NS = DP == 128 ? 5 : 8;    // tiles of the ring
  static constexpr int THREADS = 384;
  // Registers: 384 threads at 168, dealt out again by role (2 * 208 + 88 = 3 * 168).
  static constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;
  static constexpr int SMEM = 2048 + (2 + NS) * TILE;
  static constexpr uint32_t S0 = 0, O0 = 256;     // TMEM columns: S of the two tiles, O of the two
  static constexpr uint32_t TYPES = HALF ? 0u : (1u << 7) | (1u << 10);
  // fp32 accumulator, M = 128; N = 128 keys; N = DP columns, the second operand N-major
  static constexpr uint32_t IDESC_S = (1u << 4) | TYPES | ((128u >> 3) << 17) | (8u << 24);
  static constexpr uint32_t IDESC_O = (1u << 4) | TYPES | (1u << 16) | ((uint32_t)(DP >> 3) << 17) | (8u << 24);
  static constexpr float LIFT = HALF ? 7.0f : 0.0f;
};

template <int NS>
struct State {
  uint64_t full[NS], empty[NS], q_full, s_full[2], p_full[2], o_full[2];
  int32_t dead, bad;
  uint32_t tmem;
};

// The CTA's work, the same in every thread.
struct Work {
  Span w;
  int32_t t0, tp, rows;       // first token, tokens of a tile, its rows in use
  int32_t kvh, off;           // key head; key index of query 0
  int32_t kb0, n[2], step;    // first block of keys, blocks of each tile, 2: the groups share tile 0
  int32_t last;               // last token of the CTA
};

// Position in the ring of the keys and values of block b.
__device__ __forceinline__ int keys_at(int b, int step) { return step == 1 ? 2 * b : b == 0 ? 0 : 2 * b - 1; }
__device__ __forceinline__ int values_at(int b, int n, int step) {
  return step == 1 ? 2 * b + 1 : b < n - 1 ? 2 * b + 2 : 2 * n - 1;
}

// Whether some row of tokens ta .. tb does not see all of block b.
__device__ __forceinline__ bool mixed(const PromptArgs& a, const Work& x, int b, int ta, int tb) {
  const int first = (x.kb0 + b) * 128;
  return first + 128 > x.off + ta + 1 || (a.window && (int64_t)first < (int64_t)x.off + tb + 1 - a.window);
}

extern __shared__ __align__(1024) uint8_t fwd_smem[];

// Infinities and NaN of V that were cleaned away, for 32 columns of a row that sees
// keys lo .. hi - 1.
template <bool HALF>
__device__ __noinline__ void give_back(const PromptArgs& a, const Work& x, int lo, int hi, int col, float* o) {
  for (int b = 0; b < max(x.n[0], x.n[1]); ++b) {
    if (!mixed(a, x, b, x.t0, x.last)) continue;
    const int k0 = max(lo, (x.kb0 + b) * 128), k1 = min(hi, (x.kb0 + b) * 128 + 128);
    for (int k = k0; k < k1; ++k) {
      const uint16_t* v = static_cast<const uint16_t*>(a.v) + (int64_t)(x.w.k0 + k) * a.vt + x.kvh * a.vh + col;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (col + c < a.d) {
          const float f = value16<HALF>(__ldg(v + c));
          if (!isfinite(f)) o[c] += f;
        }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prompt_fwd_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.fill & CSA_FILL_OUT) {
    const int64_t words = (int64_t)a.heads * a.d / 8;
    fill_rest(a.cu_q, a.nseq, a.num_q, words, static_cast<uint4*>(a.out));
    if (a.rest) fill_rest(a.cu_q, a.nseq, a.num_q, words, static_cast<uint4*>(a.rest));
  }
  if (a.fill & CSA_FILL_LSE) fill_rest(a.cu_q, a.nseq, a.num_q, a.heads, -INFINITY, a.lse);

  // later slots first: a sequence's last tiles see the most keys
  Work x;
  const uint32_t id = gridDim.x - 1 - blockIdx.x;
  const int64_t slot = id / a.kv;
  x.kvh = (int)(id - slot * a.kv);
  x.tp = 128 / a.group;
  x.rows = x.tp * a.group;
  const int s = seq_of_slot(a.cu_q, a.nseq, 2 * x.tp, slot, lane);
  x.w = span_of(a, s);
  const int64_t local = slot - first_slot(a.cu_q, s, 2 * x.tp);
  if (local < 0 || local * 2 * x.tp >= x.w.nq) return;
  x.t0 = (int)local * 2 * x.tp;
  x.last = min(x.t0 + 2 * x.tp, x.w.nq) - 1;
  x.off = x.w.nk - x.w.nq;
  {
    const int first = a.window ? (int)max((int64_t)0, (int64_t)x.off + x.t0 + 1 - a.window) : 0;
    x.kb0 = first / 128;
    for (int t = 0; t < 2; ++t) {
      const int ta = x.t0 + t * x.tp, tb = min(ta + x.tp, x.w.nq) - 1, end = x.off + tb + 1;
      x.n[t] = tb >= ta && end > 0 ? (end + 127) / 128 - x.kb0 : 0;
    }
    x.step = 1;
    if (x.t0 + x.tp >= x.w.nq && x.n[0] > 1) {
      x.step = 2;
      x.n[1] = x.n[0];
    }
  }
  const int n = max(x.n[0], x.n[1]);

  uint8_t* const base = fwd_smem + ((1024u - (smem_at(fwd_smem) & 1023u)) & 1023u);
  auto& st = *reinterpret_cast<State<C::NS>*>(base);
  uint8_t* const q_ptr = base + 1024;
  uint8_t* const ring_ptr = q_ptr + 2 * C::TILE;
  const uint32_t q_at = smem_at(q_ptr), ring = smem_at(ring_ptr);
  const uint32_t full = smem_at(st.full), empty = smem_at(st.empty), q_full = smem_at(&st.q_full),
                 s_full = smem_at(st.s_full), p_full = smem_at(st.p_full), o_full = smem_at(st.o_full);
  volatile int32_t* const dead = &st.dead;
  if (threadIdx.x == 0) {
    st.dead = st.bad = 0;
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + 8 * t, 1);
      mbar_init(p_full + 8 * t, 4);
      mbar_init(o_full + 8 * t, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_at(&st.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&st.tmem;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 9) {  // ---- copies
      if (lane == 0 && n > 0) {
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
        const int tiles = x.step == 1 && x.n[1] > 0 ? 2 : 1;
        mbar_expect(q_full, tiles * (C::DP / 64) * 128 * x.rows);
        for (int t = 0; t < tiles; ++t)
          for (int p = 0; p < C::DP / 64; ++p)
            tma_load(q_at + t * C::TILE + p * C::SLAB, &mq, p * 64, x.kvh * a.group, x.w.q0 + x.t0 + t * x.tp, q_full);
        for (int i = 0; i < 2 * n; ++i) {
          bool value;
          int b;
          if (x.step == 1) {
            value = i & 1;
            b = i / 2;
          } else {  // K0 K1 V0 K2 V1 ...
            value = i == 2 * n - 1 || (i > 1 && (i & 1) == 0);
            b = i == 2 * n - 1 ? n - 1 : value ? i / 2 - 1 : (i + 1) / 2;
          }
          const uint32_t stage = i % C::NS;
          mbar_wait(empty + 8 * stage, ((i / C::NS) & 1) ^ 1, dead);
          if (*dead) {
            // copies under way land before the CTA ends
            for (int j = max(0, i - C::NS); j < i; ++j)
              for (int k = 0; k < kPolls && !mbar_try(full + 8 * (j % C::NS), (j / C::NS) & 1); ++k) {
              }
            for (int k = 0; k < kPolls && !mbar_try(q_full, 0); ++k) {
            }
            break;
          }
          mbar_expect(full + 8 * stage, C::TILE);
          for (int p = 0; p < C::DP / 64; ++p)
            tma_load(ring + stage * C::TILE + p * C::SLAB, value ? &mv : &mk, p * 64, x.kvh, x.w.k0 + (x.kb0 + b) * 128,
                     full + 8 * stage);
        }
      }
    } else if (warp == 8) {  // ---- matrix instructions
      if (n > 0) {
        mbar_wait(q_full, 0, dead);
        auto ready = [&](int i) { mbar_wait(full + 8 * (i % C::NS), (i / C::NS) & 1, dead); };
        auto scores = [&](int t, int b) {  // S of tile t and block b
          const uint64_t q = operand(q_at + (x.step == 1 ? t : 0) * C::TILE, 16);
          const uint64_t k = operand(ring + (keys_at(b, x.step) % C::NS) * C::TILE, 16);
  #pragma unroll
          for (int j = 0; j < C::DP / 16; ++j) {
            const int at = ((j >> 2) * C::SLAB + (j & 3) * 32) / 16;
            tc_mma(tmem + C::S0 + 128 * t, q + at, k + at, C::IDESC_S, j > 0);
          }
          tc_commit(s_full + 8 * t);
        };
        for (int t = 0; t < 2; ++t) {
          const int b = x.step == 1 ? 0 : t;
          if (x.n[t] == 0) continue;
          if (t == 0 || x.step == 2 || x.n[0] == 0) ready(keys_at(b, x.step));
          tc_after();
          __syncwarp();
          scores(t, b);
          if (x.step == 2 || t == 1 || x.n[1] == 0) tc_commit(empty + 8 * (keys_at(b, x.step) % C::NS));
        }
        const int rounds = x.step == 1 ? n : (n + 1) / 2;
        for (int r = 0; r < rounds; ++r)
          for (int t = 0; t < 2; ++t) {
            const int b = x.step == 1 ? r : 2 * r + t, next = b + x.step;
            if (b >= x.n[t]) continue;
            // step 1: tile 1 is the last to use a block, unless it has fewer (no rows)
            const bool done = x.step == 2 || t == 1 || b >= x.n[1], done_next = x.step == 2 || t == 1 || next >= x.n[1];
            const int vi = values_at(b, n, x.step);
            ready(vi);
            mbar_wait(p_full + 8 * t, r & 1, dead);
            tc_after();
            __syncwarp();
            const uint64_t v = operand(ring + (vi % C::NS) * C::TILE, C::SLAB);
  #pragma unroll
            for (int j = 0; j < 8; ++j)
              tc_mma_ts(tmem + C::O0 + C::DP * t, tmem + C::S0 + 128 * t + 8 * j, v + j * 128, C::IDESC_O, r > 0 || j > 0);
            if (done) tc_commit(empty + 8 * (vi % C::NS));
            if (next < x.n[t]) {
              ready(keys_at(next, x.step));
              tc_after();
              __syncwarp();
              scores(t, next);
              if (done_next) tc_commit(empty + 8 * (keys_at(next, x.step) % C::NS));
            } else {
              tc_commit(o_full + 8 * t);
            }
          }
      }
    }
  } else {  // ---- softmax and result: a row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + C::S0 + 128 * t, o_at = tmem + lanes + C::O0 + C::DP * t;
    const int tile = x.step == 1 ? t : 0;
    const int ta = x.t0 + tile * x.tp, tb = min(ta + x.tp, x.w.nq) - 1;
    const int token = ta + r / a.group;
    const bool there = r < x.rows && token < x.w.nq;
    const int hi = there ? x.off + token + 1 : 0;
    const int lo = a.window ? (int)max((int64_t)0, (int64_t)x.off + token + 1 - a.window) : 0;
    const float c = a.scale * kLog2e;
    float ref = -INFINITY;  // in log2 units
    float2 l0 = make_float2(0.0f, 0.0f), l1 = l0;
    int round = 0;
    for (int b = x.step == 1 ? 0 : t; b < x.n[t]; b += x.step, ++round) {
      mbar_wait(s_full + 8 * t, round & 1, dead);
      tc_after();
      if (mixed(a, x, b, x.t0, x.last)) {
        const int vi = values_at(b, n, x.step);
        mbar_wait(full + 8 * (vi % C::NS), (vi / C::NS) & 1, dead);
        clean_operand<C::HALF>(ring_ptr + (vi % C::NS) * C::TILE, C::TILE, r, 128, &st.bad);
      }
      float v[128];
#pragma unroll
      for (int k = 0; k < 4; ++k) tc_load32_async(s_at + 32 * k, v + 32 * k);
      tc_load_wait();
#pragma unroll
      for (int k = 0; k < 4; ++k) tc_loaded(v + 32 * k);
      if (mixed(a, x, b, ta, tb)) {
        const int k0 = (x.kb0 + b) * 128;
        const int h = hi - k0, w = lo - k0;
#pragma unroll
        for (int k = 0; k < 128; ++k) v[k] = k < h && k >= w ? v[k] : -INFINITY;
      }
      float m0 = fmaxf(v[0], v[1]), m1 = fmaxf(v[2], v[3]);
#pragma unroll
      for (int k = 4; k < 128; k += 4) {
        m0 = fmaxf(m0, fmaxf(v[k], v[k + 1]));
        m1 = fmaxf(m1, fmaxf(v[k + 2], v[k + 3]));
      }
      const float z = fmaxf(m0, m1) * c;
      const bool raise = z > ref + 8.0f;
      if (__any_sync(0xFFFFFFFFu, raise)) {
        const float f = raise ? ex2_approx_ftz(ref - z) : 1.0f;
        if (raise) ref = z;
        l0.x *= f;
        l0.y *= f;
        l1.x *= f;
        l1.y *= f;
        if (round > 0) {  // the products before are done: S of this block came after them
#pragma unroll 1
          for (int k = 0; k < C::DP; k += 32) {
            float o[32];
            tc_load32(o_at + k, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f;
            tc_store32(o_at + k, o);
          }
        }
      }
      const float back = C::LIFT - (ref == -INFINITY ? 0.0f : ref);
#pragma unroll
      for (int k = 0; k < 128; k += 32) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float2 za = fma2_rn(make_float2(v[k + i], v[k + i + 1]), make_float2(c, c), make_float2(back, back));
          const float2 zb = fma2_rn(make_float2(v[k + i + 2], v[k + i + 3]), make_float2(c, c), make_float2(back, back));
          const float2 pa = make_float2(ex2_approx_ftz(za.x), ex2_approx_ftz(za.y));
          const float2 pb = make_float2(ex2_approx_ftz(zb.x), ex2_approx_ftz(zb.y));
          l0 = add2_rn(l0, pa);
          l1 = add2_rn(l1, pb);
          p[i / 2] = pack16<C::HALF>(pa.x, pa.y);
          p[i / 2 + 1] = pack16<C::HALF>(pb.x, pb.y);
        }
        tc_store16_async(s_at + k / 2, p);
      }
      tc_store_wait();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * t);
    }
    float l = (l0.x + l0.y) + (l1.x + l1.y);
    if (round > 0) mbar_wait(o_full + 8 * t, 0, dead);
    tc_after();
    float f = 1.0f;  // O's factor
    if (x.step == 2) {
      // group 1's reference, sum and O by way of the ring, whose operands have all been
      // used; columns apart by 128 rows
      float* const share = reinterpret_cast<float*>(ring_ptr);
      barrier_of(1, 256);
      if (t == 1) {
        share[r] = ref;
        share[128 + r] = l;
        if (round > 0) {
#pragma unroll 1
          for (int k = 0; k < C::DP; k += 32) {
            float o[32];
            tc_load32(o_at + k, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) share[256 + (k + i) * 128 + r] = o[i];
          }
        }
      }
      barrier_of(1, 256);
      if (t == 0) {
        const float other = share[r], top = fmaxf(ref, other), safe = top == -INFINITY ? 0.0f : top;
        const float fa = ex2_approx_ftz(ref - safe), fb = ex2_approx_ftz(other - safe);
        l = l * fa + share[128 + r] * fb;
        ref = top;
#pragma unroll 1
        for (int k = 0; k < C::DP; k += 32) {
          float o[32];
          tc_load32(o_at + k, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = o[i] * fa + share[256 + (k + i) * 128 + r] * fb;
          tc_store32(o_at + k, o);
        }
      }
    }
    if (x.step == 1 || t == 0) {
      const bool some = !(l == 0.0f);
      f = some ? 1.0f / l : 0.0f;
      if (*dead) f = NAN;
      const int64_t row = (int64_t)(x.w.q0 + token) * a.heads + x.kvh * a.group + r % a.group;
      if (there) a.lse[row] = *dead ? NAN : some ? (ref - C::LIFT + log2f(l)) * kLn2 : -INFINITY;
      const bool bad = *(volatile int32_t*)&st.bad != 0;
#pragma unroll 1
      for (int k = 0; k < C::DP; k += 32) {
        float o[32];
        if (round > 0) tc_load32(o_at + k, o);
        if (!there || k >= a.d) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = some || *dead ? o[i] * f : 0.0f;
        if (round == 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = *dead ? NAN : 0.0f;
        }
        if (bad) {
          float again[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) again[i] = o[i];
          give_back<C::HALF>(a, x, lo, hi, k, again);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = again[i];
        }
        uint32_t w[16], low[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          w[i] = pack16<C::HALF>(o[2 * i], o[2 * i + 1]);
          low[i] = pack16<C::HALF>(o[2 * i] - value16<C::HALF>((uint16_t)w[i]), o[2 * i + 1] - value16<C::HALF>((uint16_t)(w[i] >> 16)));
        }
        auto put = [&](void* to, const uint32_t* v) {
          uint16_t* p = static_cast<uint16_t*>(to) + row * a.d + k;
          if (a.d % 16 == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (k + 16 * i < a.d) st_sector(p + 16 * i, v + 8 * i);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (k + 8 * i < a.d)
                *reinterpret_cast<uint4*>(p + 8 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        };
        put(a.out, w);
        if (a.rest) put(a.rest, low);
      }
    }
    tc_before();
  }
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <class C>
cudaError_t launch_fwd_of(const PromptArgs& a, cudaStream_t stream) {
  const int tp = 128 / a.group;
  const int64_t blocks = ((int64_t)a.num_q / (2 * tp) + a.nseq) * a.kv;
  CUtensorMap mq, mk, mv;
  cudaError_t e = rows_map(&mq, a.q, C::HALF, a.d, a.heads, a.num_q, a.qt, a.qh, a.group, tp);
  if (e == cudaSuccess) e = rows_map(&mk, a.k, C::HALF, a.d, a.kv, a.num_k, a.kt, a.kh, 1, 128);
  if (e == cudaSuccess) e = rows_map(&mv, a.v, C::HALF, a.d, a.kv, a.num_k, a.vt, a.vh, 1, 128);
  auto* kernel = prompt_fwd_kernel<C>;
  if (e == cudaSuccess) e = allow_dynamic_smem((const void*)kernel, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)blocks), dim3(C::THREADS), C::SMEM, stream, a, mq, mk, mv);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, bool half, cudaStream_t stream) {
  if (a.d <= 64) return half ? launch_fwd_of<Fwd<64, true>>(a, stream) : launch_fwd_of<Fwd<64, false>>(a, stream);
  return half ? launch_fwd_of<Fwd<128, true>>(a, stream) : launch_fwd_of<Fwd<128, false>>(a, stream);
}

}  // namespace csa
