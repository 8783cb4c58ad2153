// Causal attention over packed sequences, the gradient: tcgen05.
//
// Three kernels. prompt_delta_kernel reads out and grad once and writes, for each
// (token, head), lse in log2 units and delta = sum grad out - grad_lse. Then two passes
// over the pairs, each with sums of its own and in a fixed order:
//   prompt_keys_kernel, 128 keys of a key head a CTA, over the tiles of query rows
//   that see them (keys are the accumulators' lanes, so that P and dS are written
//   as first operands in tensor memory):
//     S^T = K Q^T   dP^T = V G^T   dV += P^T G   dK += dS^T Q
//   prompt_rows_kernel, 128 query rows a CTA, over the keys that they see:
//     S = Q K^T     dP = G V^T     dQ += dS K
// Seven products where one pass with atomic sums of dQ would need five; in return
// results do not depend on timing, and there is no fp32 copy of dQ to clear, add to
// and convert.
//
// In both, one warp issues the matrix instructions, one the copies, and eight warps
// form P and dS: a lane of the accumulators a thread, half of the columns each. The
// products of a tile go between the two phases of the arithmetic: keys kernel: dV of
// tile j and S of j + 1 while dS(j) is formed, dK(j) and dP(j + 1) while P(j + 1) is;
// rows kernel, where there is room for two tiles of dP: dQ(j), dP(j + 2) and S(j + 2)
// while dS(j + 1) is.
//
// fp16: P is lifted by 2^15 and dS, whose size is that of the gradients, by a power
// of two that the largest grad and v allow (prompt_delta_kernel finds them), so that
// the small ones keep their bits; bf16 needs neither.
//
// Infinities and NaN of rows that do not see the keys are cleaned from the operands
// as in the forward (csa_prompt_fwd.cu). Waits are bounded as there.
//
// What bounds it: on long sequences the tensor core under the power limit (8192 tokens of 32
// heads over 8 of 128 columns: keys kernel 700 to 735 us by the box, up to 1570 TFLOP/s of its
// four products, rows kernel 605 to 640, 1360); heads of 64 columns the arithmetic, whose
// products take half as long (8 ragged sequences of up to 1500 tokens, 24 heads over 8: 141
// and 95 us).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "csa_cache_internal.h"
#include "csa_internal.h"
#include "csa_prompt_tile.cuh"

namespace csa {

namespace {

struct BwdArgs {
  PromptArgs a;
  float2* stats;    // [num_q * heads]: -(lse log2 e - lift), -delta
  uint32_t* sizes;  // fp16: bits of the largest finite |grad row|, |v row|, |grad_lse|
  // Where items may have more than kSumTiles tiles: a place of two [DP][128] fp32 for each CTA
  // that can run, and which are taken.
  float* sums;
  uint32_t* taken;
  int32_t places;
};

// The tensor core truncates as it accumulates: 16 terms more cost up to 2^-24 of what is there,
// always towards 0 (dK of 6.4 million rows, 100003 tokens of 64 heads over one: 1.4%). So dK
// and dV leave it after this many tiles, 65536 terms, and are added up in fp32, rounded to
// nearest: less than 2^-12 is lost. A power of two.
constexpr int kSumTiles = 512;

template <bool HALF>
constexpr float kPLift = HALF ? 15.0f : 0.0f;

// fp16: |dP - delta| <= 2 |grad| |v| + |grad_lse| < 2^x, so that times 2^-x and a
// weight of at most 2^15 it stays below 2^15, in every row that is finite. bf16: x = 0.
template <bool HALF>
__device__ __forceinline__ int gradient_exponent(const BwdArgs& b) {
  if (!HALF) return 0;
  const float g = __uint_as_float(__ldg(b.sizes)), v = __uint_as_float(__ldg(b.sizes + 1)), l = __uint_as_float(__ldg(b.sizes + 2));
  const float most = fminf(fmaf(2.0f * g, v, l), 3e38f);
  if (!(most > 0.0f)) return 0;
  int x;
  frexpf(most * 1.01f, &x);
  return min(max(x, -100), 128);
}

// ---- delta -------------------------------------------------------------------

// A warp a token, for all of its heads: 8 columns a lane, so 8 or 16 lanes a head.
// fp16: further warps look at v's rows.
template <bool HALF>
__global__ void __launch_bounds__(128) prompt_delta_kernel(const __grid_constant__ BwdArgs b) {
  grid_dependency_wait();
  allow_dependent_launch();
  const PromptArgs& a = b.a;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), warps = (int64_t)gridDim.x * 4;
  const int each = a.d <= 64 ? 8 : 16, per = 32 / each;  // lanes of a head, heads of a round
  const int sub = lane / each, col = (lane % each) * 8;
  float most_g = 0.0f, most_v = 0.0f, most_l = 0.0f;
  auto total = [&](float v) {
#pragma unroll 1
    for (int o = each >> 1; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  auto at = [&](const void* base, int64_t i) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
  };
  auto unpack = [&](uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = value16<HALF>((uint16_t)w[i]);
      f[2 * i + 1] = value16<HALF>((uint16_t)(w[i] >> 16));
    }
  };
  constexpr int U = 4;  // rounds in flight
#pragma unroll 1
  for (int64_t t = id; t < a.num_q; t += warps) {
    bool in = false, single = false;
#pragma unroll 1
    for (int h0 = 0; h0 < a.heads; h0 += U * per) {
      // the loads first, of rows of no sequence too: finding the sequence takes as long
      uint4 g[U], o[U], e[U];
      float lse[U], dl[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * per + sub;
        const bool there = h < a.heads && col < a.d;
        const int64_t row = t * a.heads + h;
        g[u] = there ? at(a.g, t * a.gt + h * a.gh + col) : make_uint4(0, 0, 0, 0);
        o[u] = there ? at(a.out, row * a.d + col) : make_uint4(0, 0, 0, 0);
        e[u] = there && a.rest ? at(a.rest, row * a.d + col) : make_uint4(0, 0, 0, 0);
        lse[u] = there ? __ldg(a.lse + row) : 0.0f;
        dl[u] = there && a.grad_lse ? __ldg(a.grad_lse + row) : 0.0f;
      }
      if (h0 == 0) {
        // the token's sequence: the last one that begins at or before it
        int lo = 0, span = a.nseq;
#pragma unroll 1
        while (span > 1) {
          const int step = (span + 31) / 32, first = lo + lane * step;
          const bool before = lane * step < span && __ldg(a.cu_q + first) <= t;
          const unsigned who = __ballot_sync(0xFFFFFFFFu, before);
          const int k = who ? 31 - __clz(who) : 0;
          span = min(step, span - k * step);
          lo += k * step;
        }
        const Span w = span_of<false>(a, lo);
        in = t >= w.q0 && t < (int64_t)w.q0 + w.nq;
        single = in && (a.window == 1 || w.nk - w.nq + (int)(t - w.q0) + 1 == 1);
        if (!in) break;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * per + sub;
        float x[8], y[8], z[8], dot = 0.0f, size = 0.0f;
        unpack(g[u], x);
        unpack(o[u], y);
        unpack(e[u], z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = fmaf(x[i], z[i], fmaf(x[i], y[i], dot));
          size = fmaf(x[i], x[i], size);
        }
        // A gradient that is not finite has NaN for its delta: dP is formed of operands that the
        // keys kernel may be cleaning, and whatever it is then, dS is NaN for all keys that the row sees.
        if (infinite_bits<HALF>(g[u])) dot = NAN;
        dot = total(dot);
        if (HALF) size = total(size);
        if (h < a.heads && lane % each == 0) {
          b.stats[t * a.heads + h] =
              make_float2(lse[u] == -INFINITY ? -INFINITY : kPLift<HALF> - lse[u] * kLog2e, single ? dl[u] : dl[u] - dot);
          // Rows that are not finite stay so whatever the scale, through delta, and those that see
          // no key have no weight: a scale for either would be the other rows' loss.
          if (HALF && lse[u] != -INFINITY) {
            const float s = sqrtf(size);
            if (isfinite(s)) most_g = fmaxf(most_g, s);
            if (isfinite(dl[u])) most_l = fmaxf(most_l, fabsf(dl[u]));
          }
        }
      }
    }
  }
  if (HALF) {
    // rows of no sequence may hold anything
    const int64_t k1 = min(__ldg(a.cu_k + a.nseq), a.num_k);
#pragma unroll 1
    for (int64_t t = max(__ldg(a.cu_k), 0) + id; t < k1; t += warps)
#pragma unroll 1
      for (int h0 = 0; h0 < a.kv; h0 += per) {
        const int h = h0 + sub;
        float size = 0.0f;
        if (h < a.kv && col < a.d) {
          float v[8];
          unpack(at(a.v, t * a.vt + h * a.vh + col), v);
#pragma unroll
          for (int i = 0; i < 8; ++i) size = isfinite(v[i]) ? fmaf(v[i], v[i], size) : size;
        }
        size = sqrtf(total(size));
        most_v = fmaxf(most_v, size);
      }
    const uint32_t g = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most_g));
    const uint32_t v = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most_v));
    const uint32_t l = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most_l));
    if (lane == 0) {  // a look first: few of the warps have the largest so far
      volatile uint32_t* const sizes = b.sizes;
      if (g > sizes[0]) atomicMax(b.sizes, g);
      if (v > sizes[1]) atomicMax(b.sizes + 1, v);
      if (l > sizes[2]) atomicMax(b.sizes + 2, l);
    }
  }
}

// ---- what both passes share ---------------------------------------------------

template <int DP_, bool HALF_>
struct Bwd {
  static constexpr int DP = DP_;
  static constexpr bool HALF = HALF_;
  static constexpr int SLAB = 16384;
  static constexpr int TILE = DP / 64 * SLAB;
  static constexpr int HEAD = 8192;  // barriers and the rows' numbers
  static constexpr int THREADS = 384;
  static constexpr int MATH_REGS = 208, OTHER_REGS = 88;  // 2 * 208 + 88 = 3 * 168
  static constexpr uint32_t TYPES = HALF ? 0u : (1u << 7) | (1u << 10);
  // both operands K-major, N = 128; the second N-major, N = DP
  static constexpr uint32_t IDESC_S = (1u << 4) | TYPES | ((128u >> 3) << 17) | (8u << 24);
  static constexpr uint32_t IDESC_D = (1u << 4) | TYPES | (1u << 16) | ((uint32_t)(DP >> 3) << 17) | (8u << 24);
};

extern __shared__ __align__(1024) uint8_t bwd_smem[];

// D [128 x 128] = A B^T over the columns of two operands in shared memory.
template <class C>
__device__ __forceinline__ void product(uint32_t leader, uint32_t d, uint32_t a, uint32_t b) {
  const uint64_t x = operand(a, 16), y = operand(b, 16);
#pragma unroll
  for (int p = 0; p < C::DP / 64; ++p) tc_mma4<2>(leader, d, x + p * (C::SLAB / 16), y + p * (C::SLAB / 16), C::IDESC_S, p > 0);
}
// D [128 x DP] += A B, A in tensor memory, the 16-bit weights of 64 of the 128 at `a`,
// in the place of the logits that they were formed from; half: which 64.
template <class C>
__device__ __forceinline__ void product_add(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, int half, bool add) {
  tc_mma4_ts<128>(leader, d, a + 64 * half, operand(b, C::SLAB) + 512 * half, C::IDESC_D, add);
}

// 32 values of a lane as 16 words of tensor memory, without waiting.
template <bool HALF>
__device__ __forceinline__ void store_part(uint32_t at, const float* v) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack16<HALF>(v[2 * i], v[2 * i + 1]);
  tc_store16_async(at, w);
}

// 32 columns of a row of a result.
template <bool HALF>
__device__ __forceinline__ void store_columns(void* to, int64_t at, int d, int col, const float* v) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack16<HALF>(v[2 * i], v[2 * i + 1]);
  uint16_t* p = static_cast<uint16_t*>(to) + at + col;
  if (reinterpret_cast<uintptr_t>(p) % 32 == 0 && d % 16 == 0) {  // tensors are 16-byte aligned at least
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (col + 16 * i < d) st_sector(p + 16 * i, w + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + 8 * i < d) *reinterpret_cast<uint4*>(p + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

template <class C>
__device__ __forceinline__ void load_tile(uint32_t to, const CUtensorMap* map, int head, int token, uint32_t bar) {
#pragma unroll 1
  for (int p = 0; p < C::DP / 64; ++p) tma_load(to + p * C::SLAB, map, p * 64, head, token, bar);
}

// ---- dK and dV ----------------------------------------------------------------

struct alignas(16) KeysItem {
  Span w;
  int32_t k0, kvh, off;  // first key within the sequence; key head; key index of query 0
  int32_t t0, tp, n0;    // first query token, tokens of a tile, tiles
  int32_t pad[2];
  __device__ __forceinline__ bool keys() const { return n0 > 0; }
};

struct KeysState {
  alignas(16) float lse[2][128];    // of a tile's rows: -(lse log2 e - lift)
  alignas(16) float delta[2][128];  // -delta, times 2^-x for fp16
  alignas(16) int32_t lo[2][128];   // keys that they see
  alignas(16) int32_t hi[2][128];
  KeysItem item[2];
  WorkState work;
  uint64_t kv_full, kv_empty, q_full[2], q_empty[2], g_full[2], g_empty[2], r_full[2], s_full, p_full[2], dp_full, ds_full[2], done, clean[2];
  int32_t dead, bad;
  uint32_t tmem;
  int32_t place;  // of BwdArgs::sums
};
static_assert(sizeof(KeysState) <= 8192, "HEAD");

// Item `id`, by a warp; n0 < 0 where the slot has none. Earlier slots first: a sequence's
// first keys are seen by the most rows.
__device__ __forceinline__ KeysItem keys_item(const PromptArgs& a, uint32_t id, int lane) {
  KeysItem x;
  const int64_t slot = id / a.kv;
  x.kvh = (int)(id - slot * a.kv);
  const int s = seq_of_slot(a.cu_k, a.nseq, 128, slot, lane);
  x.w = span_of<true>(a, s);
  x.n0 = -1;
  const int64_t local = slot - first_slot(a.cu_k, s, 128);
  if (local < 0 || local * 128 >= x.w.nk) return x;
  x.k0 = (int)local * 128;
  x.off = x.w.nk - x.w.nq;
  x.tp = 128 / a.group;
  x.t0 = max(0, x.k0 - x.off);
  int t1 = x.w.nq;  // behind the last query that sees a key
  if (a.window) t1 = (int)min((int64_t)t1, (int64_t)min(x.k0 + 128, x.w.nk) - 1 - x.off + a.window);
  x.n0 = t1 > x.t0 ? (t1 - x.t0 + x.tp - 1) / x.tp : 0;
  return x;
}

// Whether some row of tile j does not see some key of the CTA, or is not there.
__device__ __forceinline__ bool keys_mixed(const PromptArgs& a, const KeysItem& x, int j) {
  const int64_t ta = (int64_t)x.t0 + (int64_t)j * x.tp, tb = ta + x.tp - 1;
  return x.k0 + 128 > x.off + ta + 1 || tb >= x.w.nq || (a.window && x.k0 < x.off + tb + 1 - a.window);
}

// Infinities and NaN of grad that were cleaned away, for 32 columns of a key's dv.
template <bool HALF>
__device__ __noinline__ void give_back_grad(const PromptArgs& a, const KeysItem& x, int key, int col, float* o) {
#pragma unroll 1
  for (int j = 0; j < x.n0; ++j) {
    if (!keys_mixed(a, x, j)) continue;
#pragma unroll 1
    for (int i = 0; i < x.tp; ++i) {
      const int t = x.t0 + j * x.tp + i;
      const int64_t hi = (int64_t)x.off + t + 1;
      if (t >= x.w.nq || key >= hi || (a.window && key < hi - a.window)) continue;
#pragma unroll 1
      for (int h = x.kvh * a.group; h < (x.kvh + 1) * a.group; ++h) {
        const uint16_t* g = static_cast<const uint16_t*>(a.g) + (int64_t)(x.w.q0 + t) * a.gt + h * a.gh + col;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (col + c < a.d) {
            const float f = value16<HALF>(__ldg(g + c));
            if (!isfinite(f)) o[c] += f;
          }
      }
    }
  }
}

// What the arithmetic of the keys kernel's tiles needs.
struct KeysMath {
  Dead dead;
  uint32_t s_at, dp_at, r_full, s_full, p_full, dp_full, ds_full;
  int col, key;
  float c, f;
};

// P and dS of the CTA's j-th tile for a key and 64 rows; SOME: some row does not see some key;
// says whether some key of the warp has NaN for the last row's logit. In two parts of 32 rows: the second's logits arrive while the first's are used.
template <class C, bool SOME>
__device__ __forceinline__ bool keys_step(KeysState& st, const KeysMath& m, uint32_t j) {
  constexpr bool HALF = C::HALF;
  const int stage = j & 1, key = m.key, lane = threadIdx.x & 31;
  const float2 c2 = make_float2(m.c, m.c), f2 = make_float2(m.f, m.f);
  wait_for(m.r_full + 8 * stage, (j >> 1) & 1, m.dead);
  wait_for(m.s_full, j & 1, m.dead);
  tc_after();
  float p[64], d[64];
  bool nan = false;
  tc_load32_async(m.s_at, p);
  tc_load_wait();
  tc_loaded(p);
  tc_load32_async(m.s_at + 32, p + 32);
#pragma unroll
  for (int part = 0; part < 64; part += 32) {
    if (part) {
      tc_load_wait();
      tc_loaded(p + 32);
      if constexpr (SOME) nan = p[63] != p[63];
    }
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const int k = part + i;
      const float4 l = *reinterpret_cast<const float4*>(&st.lse[stage][m.col + k]);
      const float2 za = fma2_rn(make_float2(p[k], p[k + 1]), c2, make_float2(l.x, l.y));
      const float2 zb = fma2_rn(make_float2(p[k + 2], p[k + 3]), c2, make_float2(l.z, l.w));
      p[k] = ex2_approx_ftz(za.x);
      p[k + 1] = ex2_approx_ftz(za.y);
      p[k + 2] = ex2_approx_ftz(zb.x);
      p[k + 3] = ex2_approx_ftz(zb.y);
      if constexpr (SOME) {
        const int4 lo = *reinterpret_cast<const int4*>(&st.lo[stage][m.col + k]), hi = *reinterpret_cast<const int4*>(&st.hi[stage][m.col + k]);
        p[k] = key >= lo.x && key < hi.x ? p[k] : 0.0f;
        p[k + 1] = key >= lo.y && key < hi.y ? p[k + 1] : 0.0f;
        p[k + 2] = key >= lo.z && key < hi.z ? p[k + 2] : 0.0f;
        p[k + 3] = key >= lo.w && key < hi.w ? p[k + 3] : 0.0f;
      }
    }
    store_part<HALF>(m.s_at + part / 2, p + part);
  }
  tc_store_wait();
  tc_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(m.p_full);

  wait_for(m.dp_full, j & 1, m.dead);
  tc_after();
  tc_load32_async(m.dp_at, d);
  tc_load_wait();
  tc_loaded(d);
  tc_load32_async(m.dp_at + 32, d + 32);
#pragma unroll
  for (int part = 0; part < 64; part += 32) {
    if (part) {
      tc_load_wait();
      tc_loaded(d + 32);
    }
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const int k = part + i;
      const float4 l = *reinterpret_cast<const float4*>(&st.delta[stage][m.col + k]);
      float2 da, db;
      if constexpr (HALF) {
        da = fma2_rn(make_float2(d[k], d[k + 1]), f2, make_float2(l.x, l.y));
        db = fma2_rn(make_float2(d[k + 2], d[k + 3]), f2, make_float2(l.z, l.w));
      } else {
        da = add2_rn(make_float2(d[k], d[k + 1]), make_float2(l.x, l.y));
        db = add2_rn(make_float2(d[k + 2], d[k + 3]), make_float2(l.z, l.w));
      }
      if constexpr (SOME) {  // rows that see one key: dP does not count; rows that see none of it: nothing does
        const int4 lo = *reinterpret_cast<const int4*>(&st.lo[stage][m.col + k]), hi = *reinterpret_cast<const int4*>(&st.hi[stage][m.col + k]);
        da.x = hi.x - lo.x == 1 ? l.x : da.x;
        da.y = hi.y - lo.y == 1 ? l.y : da.y;
        db.x = hi.z - lo.z == 1 ? l.z : db.x;
        db.y = hi.w - lo.w == 1 ? l.w : db.y;
        da.x = key >= lo.x && key < hi.x ? da.x : 0.0f;
        da.y = key >= lo.y && key < hi.y ? da.y : 0.0f;
        db.x = key >= lo.z && key < hi.z ? db.x : 0.0f;
        db.y = key >= lo.w && key < hi.w ? db.y : 0.0f;
      }
      const float2 sa = mul2_rn(make_float2(p[k], p[k + 1]), da), sb = mul2_rn(make_float2(p[k + 2], p[k + 3]), db);
      d[k] = sa.x;
      d[k + 1] = sa.y;
      d[k + 2] = sb.x;
      d[k + 3] = sb.y;
    }
    store_part<HALF>(m.dp_at + part / 2, d + part);
  }
  tc_store_wait();
  tc_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(m.ds_full);
  return SOME && __any_sync(0xFFFFFFFFu, nan);
}
// Kept out of the loop: with both forms in it the instruction cache held neither
// (8192 tokens of 32 heads of 128: 875 us).
template <class C>
__device__ __noinline__ bool keys_step_some(KeysState& st, const KeysMath& m, uint32_t j) {
  return keys_step<C, true>(st, m, j);
}

// The sums of a stretch of tiles, added to what the stretches before left: a key a thread.
template <class C>
__device__ __noinline__ void set_aside(float* sums, uint32_t at, bool first) {
#pragma unroll 1
  for (int i = 0; i < C::DP; i += 32) {
    float o[32];
    tc_load32(at + i, o);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      float* const to = sums + (i + c) * 128;
      *to = first ? o[c] : *to + o[c];
    }
  }
  tc_before();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prompt_keys_kernel(const __grid_constant__ BwdArgs b, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mg) {
  grid_dependency_wait();
  allow_dependent_launch();
  const PromptArgs& a = b.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tp = 128 / a.group, rows = tp * a.group;
  uint8_t* const base = bwd_smem + ((1024u - (smem_at(bwd_smem) & 1023u)) & 1023u);
  auto& st = *reinterpret_cast<KeysState*>(base);
  uint8_t* const q_ptr = base + C::HEAD + 2 * C::TILE;
  uint8_t* const g_ptr = q_ptr + 2 * C::TILE;
  const uint32_t k_at = smem_at(base + C::HEAD), v_at = k_at + C::TILE, q_at = smem_at(q_ptr), g_at = smem_at(g_ptr);
  const uint32_t kv_full = smem_at(&st.kv_full), kv_empty = smem_at(&st.kv_empty), q_full = smem_at(st.q_full),
                 q_empty = smem_at(st.q_empty), g_full = smem_at(st.g_full), g_empty = smem_at(st.g_empty),
                 r_full = smem_at(st.r_full), s_full = smem_at(&st.s_full), p_full = smem_at(st.p_full),
                 dp_full = smem_at(&st.dp_full), ds_full = smem_at(st.ds_full), done = smem_at(&st.done),
                 clean = smem_at(st.clean);
  const Dead dead = {&st.dead, a.polls};
  if (threadIdx.x == 0) {
    st.dead = st.bad = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(clean + 8 * i, 1);
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(g_full + 8 * i, 1);
      mbar_init(g_empty + 8 * i, 1);
      mbar_init(r_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(ds_full + 8 * i, 4);
    }
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(done, 1);
    init_work(st.work, 11);  // eight warps of the arithmetic, copies, the rows' numbers, matrix instructions
    if (b.sums) {  // as many places as CTAs reside, so that one is free
      uint32_t sm;
      asm("mov.u32 %0, %smid;" : "=r"(sm));
      int place = (int)(sm % (uint32_t)b.places);
#pragma unroll 1
      for (int i = 0; atomicExch(b.taken + place, 1u); ++i) {
        place = place + 1 < b.places ? place + 1 : 0;
        if (i == kPolls) {
          st.dead = 1;
          break;
        }
      }
      st.place = place;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows of a tile that no head uses are never copied to, and must not hold NaN
  if (rows < 128) {
#pragma unroll 1
    for (int i = threadIdx.x; i < 4 * (C::DP / 64) * (128 - rows) * 8; i += C::THREADS) {
      const int slab = i / ((128 - rows) * 8), at = i - slab * (128 - rows) * 8;
      *reinterpret_cast<uint4*>(q_ptr + slab * C::SLAB + rows * 128 + at * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_at(&st.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&st.tmem;
  auto take = [&](int k) { return take_work(st.work, st.item, k, lane, dead); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 11) {  // ---- work
      find_work(st.work, st.item, blockIdx.x, false, lane, dead, [&](uint32_t id) {
        const int64_t words = (int64_t)a.kv * a.d / 8, from = (int64_t)id * 32 + lane, step = (int64_t)gridDim.x * 32;
        fill_rest(a.cu_k, a.nseq, a.num_k, words, static_cast<uint4*>(a.dk), from, step);
        fill_rest(a.cu_k, a.nseq, a.num_k, words, static_cast<uint4*>(a.dv), from, step);
        return keys_item(a, id, lane);
      });
    } else if (warp == 9) {  // ---- copies
      uint32_t q_tiles = 0, g_tiles = 0, loaded = 0;
      const int bytes = C::DP / 64 * 128 * rows;
#pragma unroll 1
      for (int k = 0;; ++k) {
        const KeysItem x = take(k);
        if (x.n0 < 0) break;
        if (x.n0 == 0) continue;
        if (lane == 0) wait_for(kv_empty, (loaded & 1) ^ 1, dead);
        if (lane == 0 && !*dead) {
          ++loaded;
          mbar_expect(kv_full, 2 * C::TILE);
          load_tile<C>(k_at, &mk, x.kvh, x.w.k0 + x.k0, kv_full);
          load_tile<C>(v_at, &mv, x.kvh, x.w.k0 + x.k0, kv_full);
#pragma unroll 1
          for (int j = 0; j < x.n0; ++j) {
            const uint32_t stage = q_tiles & 1, parity = ((q_tiles >> 1) & 1) ^ 1;
            const int token = x.w.q0 + x.t0 + j * tp;
            wait_for(q_empty + 8 * stage, parity, dead);
            if (*dead) break;
            ++q_tiles;
            mbar_expect(q_full + 8 * stage, bytes);
            load_tile<C>(q_at + stage * C::TILE, &mq, x.kvh * a.group, token, q_full + 8 * stage);
            wait_for(g_empty + 8 * stage, parity, dead);
            if (*dead) break;
            ++g_tiles;
            mbar_expect(g_full + 8 * stage, bytes);
            load_tile<C>(g_at + stage * C::TILE, &mg, x.kvh * a.group, token, g_full + 8 * stage);
          }
        }
        __syncwarp();
      }
      if (lane == 0) {
        land_ring(kv_full, 1, loaded);
        land_ring(q_full, 2, q_tiles);
        land_ring(g_full, 2, g_tiles);
      }
    } else if (warp == 10) {  // ---- the rows' numbers, with the tile of q; cleaning
      // S and dP of a tile may be formed before, while or after it is cleaned: a row that holds
      // infinities has lse or delta to match (-inf where all its logits are, NaN otherwise), which
      // makes P and dS the same either way. dV and dK wait for clean operands.
      const float f = C::HALF ? exp2f((float)-gradient_exponent<C::HALF>(b)) : 1.0f;
      uint32_t tiles = 0;
      int token[4], head[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        token[i] = (i * 32 + lane) / a.group;
        head[i] = i * 32 + lane - token[i] * a.group;
      }
#pragma unroll 1
      for (int k = 0;; ++k) {
        const KeysItem x = take(k);
        if (x.n0 < 0) break;
#pragma unroll 1
        for (int j = 0; j < x.n0; ++j, ++tiles) {
          const uint32_t stage = tiles & 1;
          float2 v[4];
          int hi[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = x.t0 + j * tp + token[i];
            const bool there = i * 32 + lane < rows && t < x.w.nq;
            hi[i] = there ? x.off + t + 1 : 0;
            v[i] = there ? __ldg(b.stats + (int64_t)(x.w.q0 + t) * a.heads + x.kvh * a.group + head[i]) : make_float2(-INFINITY, 0.0f);
          }
          wait_for(q_empty + 8 * stage, ((tiles >> 1) & 1) ^ 1, dead);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 32 + lane;
            st.lse[stage][r] = v[i].x;
            st.delta[stage][r] = v[i].y * f;
            st.hi[stage][r] = hi[i];
            st.lo[stage][r] = a.window ? max(0, hi[i] - a.window) : 0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(r_full + 8 * stage);
          tile_seen(st.work, lane);
          if (keys_mixed(a, x, j)) {  // infinities and NaN of rows that do not see every key
            const uint32_t parity = (tiles >> 1) & 1;
            wait_for(q_full + 8 * stage, parity, dead);
            clean_operand<C::HALF>(q_ptr + stage * C::TILE, C::TILE, lane, &st.bad);
            wait_for(g_full + 8 * stage, parity, dead);
            clean_operand<C::HALF>(g_ptr + stage * C::TILE, C::TILE, lane, &st.bad);
            __syncwarp();
            if (lane == 0) mbar_arrive(clean + 8 * stage);
          }
        }
      }
    } else if (warp == 8) {  // ---- matrix instructions
      const uint32_t leader = tc_leader(), tm = uniform(tmem), S = tm, DP = tm + 128, DV = tm + 256, DK = tm + 256 + C::DP;
      uint32_t tiles = 0, items = 0, cleaned = 0;  // cleaned: a parity a stage
      auto scores = [&](uint32_t j) {
        wait_for(q_full + 8 * (j & 1), (j >> 1) & 1, dead);
        tc_after();
        product<C>(leader, S, k_at, q_at + (j & 1) * C::TILE);
        tc_commit_by(leader, s_full);
      };
      auto weights = [&](uint32_t j) {  // dP
        wait_for(g_full + 8 * (j & 1), (j >> 1) & 1, dead);
        tc_after();
        product<C>(leader, DP, v_at, g_at + (j & 1) * C::TILE);
        tc_commit_by(leader, dp_full);
      };
      auto add = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t ready, uint32_t j, bool first) {
        // The first product of an item, or of a stretch, writes over the last one's sums: both
        // groups of the arithmetic have read them when both have formed something of this one.
        if (first) wait_for(ready + 8, j & 1, dead);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait_for(ready + 8 * half, j & 1, dead);
          tc_after();
          product_add<C>(leader, d, x, y, half, !first || half > 0);
        }
      };
#pragma unroll 1
      for (int k = 0;; ++k) {
        const KeysItem x = take(k);
        const int n = (int)uniform((uint32_t)x.n0);
        if (n < 0) break;
        if (n == 0) continue;
        wait_for(kv_full, items & 1, dead);
        ++items;
        scores(tiles);
        weights(tiles);
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++tiles) {
          if (j == max(0, n - 3)) want_work(st.work, lane);
          if (keys_mixed(a, x, j)) {
            wait_for(clean + 8 * (tiles & 1), (cleaned >> (tiles & 1)) & 1, dead);
            cleaned ^= 1u << (tiles & 1);
            tc_after();
          }
          const bool first = (j & (kSumTiles - 1)) == 0;
          add(DV, S, g_at + (tiles & 1) * C::TILE, p_full, tiles, first);
          tc_commit_by(leader, g_empty + 8 * (tiles & 1));
          if (j + 1 < n) scores(tiles + 1);
          add(DK, DP, q_at + (tiles & 1) * C::TILE, ds_full, tiles, first);
          tc_commit_by(leader, q_empty + 8 * (tiles & 1));
          if (((j + 1) & (kSumTiles - 1)) == 0 && j + 1 < n) tc_commit_by(leader, done);
          if (j + 1 < n)
            weights(tiles + 1);
          else
            tc_commit_by(leader, kv_empty);
        }
        tc_commit_by(leader, done);
      }
      end_products(st.work, leader);
    }
  } else {  // ---- P and dS: a key a thread, half of a tile's rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MATH_REGS));
    const int half = warp >> 2, col = half * 64;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int e = gradient_exponent<C::HALF>(b);
    KeysMath m = {dead, tmem + lanes + col, tmem + 128 + lanes + col, r_full, s_full, p_full + 8 * half, dp_full,
                  ds_full + 8 * half, col, 0, a.scale * kLog2e, C::HALF ? exp2f((float)-e) : 1.0f};
    uint32_t tiles = 0, stretches = 0;
    // this thread's of the CTA's place
    float* const sums = b.sums + ((int64_t)(b.sums ? st.place : 0) * 2 + half) * C::DP * 128 + (threadIdx.x & 127);
#pragma unroll 1
    for (int k = 0;; ++k) {
      KeysItem x = take(k);
      if (x.n0 < 0) break;
      m.key = x.k0 + (threadIdx.x & 127);
      const int32_t nq = x.w.nq;
      // Rows that no head uses, behind the 64th, are 0: a key that holds infinities has NaN for
      // their logits. The first tile, masked as mixed ones are (nq 0), says so, and all are then.
      if (half && rows < 128) x.w.nq = 0;
#pragma unroll 1
      for (int j = 0; j < x.n0;) {  // stretches
        const int end = min(x.n0, j + kSumTiles);
#pragma unroll 1
        for (; j < end; ++j, ++tiles) {
          if (keys_mixed(a, x, j)) {
            const bool nan = keys_step_some<C>(st, m, tiles);
            if (j == 0 && !nan) x.w.nq = nq;
          } else {
            keys_step<C, false>(st, m, tiles);
          }
        }
        if (j < x.n0) {
          wait_for(done, stretches++ & 1, dead);
          tc_after();
          set_aside<C>(sums, tmem + 256 + half * C::DP + lanes, j <= kSumTiles);
        }
      }
      x.w.nq = nq;
      // group 0 stores dV, group 1 dK
      if (x.n0 > 0) wait_for(done, stretches++ & 1, dead);
      tc_after();
      const bool there = m.key < x.w.nk;
      const int64_t row = ((int64_t)(x.w.k0 + m.key) * a.kv + x.kvh) * a.d;
      float factor = half ? a.scale * (C::HALF ? exp2f((float)(e - 15)) : 1.0f) : (C::HALF ? exp2f(-15.0f) : 1.0f);
      if (*dead) factor = NAN;
      // cleaned before the products that `done` stands for
      const bool bad = half == 0 && *(volatile int32_t*)&st.bad != 0;
#pragma unroll 1
      for (int i = 0; i < C::DP; i += 32) {
        float o[32];
        if (x.n0 > 0) tc_load32(tmem + 256 + half * C::DP + lanes + i, o);
        if (x.n0 > kSumTiles) {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] += sums[(i + c) * 128];
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = x.n0 > 0 ? o[c] * factor : 0.0f;
        if (bad && there && i < a.d) {
          float again[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) again[c] = o[c];
          give_back_grad<C::HALF>(a, x, m.key, i, again);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = again[c];
        }
        if (there && i < a.d) store_columns<C::HALF>(half ? a.dk : a.dv, row, a.d, i, o);
      }
      tc_before();
    }
  }
  __syncwarp();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (b.sums && threadIdx.x == 0) {
    __threadfence();
    atomicExch(b.taken + st.place, 0u);
  }
  if (*dead)
    for_last_items(st.work, [&](uint32_t id) {
      const KeysItem x = keys_item(a, id, lane);
      const int vectors = a.d / 8;
#pragma unroll 1
      for (int i = threadIdx.x; i < min(128, x.w.nk - x.k0) * vectors; i += C::THREADS) {
        const int64_t row = (int64_t)(x.w.k0 + x.k0 + i / vectors) * a.kv + x.kvh;
        put_nan(a.dk, row, vectors, i % vectors);
        put_nan(a.dv, row, vectors, i % vectors);
      }
    });
}

// ---- dQ -------------------------------------------------------------------------

constexpr int kKeyStages = 3, kValueStages = 2;

struct alignas(16) RowsItem {
  Span w;
  int32_t t0, t1, kvh, off;  // tokens t0 .. t1 - 1; key head; key index of query 0
  int32_t kb0, n0;           // first block of keys, blocks
  int32_t pad[2];
  __device__ __forceinline__ bool keys() const { return n0 > 0; }
};

struct RowsState {
  RowsItem item[2];
  WorkState work;
  uint64_t q_full, q_empty, k_full[kKeyStages], k_empty[kKeyStages], v_full[kValueStages], v_empty[kValueStages], clean[kKeyStages], scored[kKeyStages],
      s_full, s_empty, dp_full[2], ds_full[2][2], done;  // ds_full: the arithmetic may be a block ahead
  int32_t dead, bad;
  uint32_t tmem;
};
static_assert(sizeof(RowsState) <= 1024, "in front of the tiles");

// Item `id`, by a warp; n0 < 0 where the slot has none. Later slots first: a sequence's last
// tiles see the most keys.
__device__ __forceinline__ RowsItem rows_item(const PromptArgs& a, uint32_t id, uint32_t ids, int lane) {
  RowsItem x;
  const int tp = 128 / a.group;
  id = ids - 1 - id;
  const int64_t slot = id / a.kv;
  x.kvh = (int)(id - slot * a.kv);
  const int s = seq_of_slot(a.cu_q, a.nseq, tp, slot, lane);
  x.w = span_of<false>(a, s);
  x.n0 = -1;
  const int64_t local = slot - first_slot(a.cu_q, s, tp);
  if (local < 0 || local * tp >= x.w.nq) return x;
  x.t0 = (int)local * tp;
  x.t1 = min(x.t0 + tp, x.w.nq);
  x.off = x.w.nk - x.w.nq;
  x.kb0 = (a.window ? (int)max((int64_t)0, (int64_t)x.off + x.t0 + 1 - a.window) : 0) / 128;
  x.n0 = x.off + x.t1 > 0 ? (x.off + x.t1 + 127) / 128 - x.kb0 : 0;
  return x;
}

// Whether some row of the item does not see some key of block j.
__device__ __forceinline__ bool rows_mixed(const PromptArgs& a, const RowsItem& x, int j) {
  const int first = (x.kb0 + j) * 128;
  return first + 128 > x.off + x.t0 + 1 || (a.window && (int64_t)first < (int64_t)x.off + x.t1 - a.window);
}

// The blocks [from, to) for which that does not hold.
__device__ __forceinline__ int2 rows_whole(const PromptArgs& a, const RowsItem& x) {
  const int64_t from = a.window ? ((int64_t)x.off + x.t1 - a.window + 127) >> 7 : 0;
  return make_int2((int)max(from - x.kb0, (int64_t)0), max(x.off + x.t0 + 1, 0) / 128 - x.kb0);
}

// What the arithmetic of a row's blocks needs.
struct RowsMath {
  Dead dead;
  uint32_t s_at, dp_at, s_full, s_empty, dp_full, ds_full;
  int lo, hi;  // keys that the row sees, from this thread's half of block 0 on
  bool single;
  float c, f, lse, delta;
};

// dS of the CTA's j-th block for a row and 64 keys, the first of them `first` behind the
// item's first; SOME: some row does not see some key.
template <class C, bool SOME>
__device__ __forceinline__ void rows_step(const RowsMath& m, uint32_t j, int first) {
  const int lane = threadIdx.x & 31;
  const float2 c2 = make_float2(m.c, m.c), f2 = make_float2(m.f, m.f), l2 = make_float2(m.lse, m.lse),
               d2 = make_float2(m.delta, m.delta);
  const uint32_t dp_at = m.dp_at + 128 * (j & 1);
  wait_for(m.s_full, j & 1, m.dead);
  tc_after();
  float p[64], d[64];
  tc_load32_async(m.s_at, p);
  tc_load32_async(m.s_at + 32, p + 32);
  tc_load_wait();
  tc_loaded(p);
  tc_loaded(p + 32);
  tc_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(m.s_empty);
#pragma unroll
  for (int k = 0; k < 64; k += 2) {
    const float2 z = fma2_rn(make_float2(p[k], p[k + 1]), c2, l2);
    p[k] = ex2_approx_ftz(z.x);
    p[k + 1] = ex2_approx_ftz(z.y);
  }
  wait_for(m.dp_full + 8 * (j & 1), (j >> 1) & 1, m.dead);
  tc_after();
  tc_load32_async(dp_at, d);
  tc_load_wait();
  tc_loaded(d);
  tc_load32_async(dp_at + 32, d + 32);
#pragma unroll
  for (int part = 0; part < 64; part += 32) {
    if (part) {
      tc_load_wait();
      tc_loaded(d + 32);
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const int k = part + i;
      float2 v = make_float2(d[k], d[k + 1]);
      if constexpr (C::HALF)
        v = fma2_rn(v, f2, d2);
      else
        v = add2_rn(v, d2);
      if constexpr (SOME) {
        if (m.single) v = d2;  // a row that sees one key: dP does not count
      }
      v = mul2_rn(make_float2(p[k], p[k + 1]), v);
      d[k] = v.x;
      d[k + 1] = v.y;
      if constexpr (SOME) {
        d[k] = first + k < m.hi && first + k >= m.lo ? d[k] : 0.0f;
        d[k + 1] = first + k + 1 < m.hi && first + k + 1 >= m.lo ? d[k + 1] : 0.0f;
      }
    }
    store_part<C::HALF>(dp_at + part / 2, d + part);
  }
  tc_store_wait();
  tc_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(m.ds_full + 16 * (j & 1));
}
template <class C>
__device__ __noinline__ void rows_step_some(const RowsMath& m, uint32_t j, int first) {
  rows_step<C, true>(m, j, first);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prompt_rows_kernel(const __grid_constant__ BwdArgs b, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mg) {
  grid_dependency_wait();
  allow_dependent_launch();
  const PromptArgs& a = b.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tp = 128 / a.group, rows = tp * a.group;
  uint8_t* const base = bwd_smem + ((1024u - (smem_at(bwd_smem) & 1023u)) & 1023u);
  auto& st = *reinterpret_cast<RowsState*>(base);
  uint8_t* const k_ptr = base + 1024 + 2 * C::TILE;
  const uint32_t q_at = smem_at(base + 1024), g_at = q_at + C::TILE, k_at = smem_at(k_ptr), v_at = k_at + kKeyStages * C::TILE;
  const uint32_t q_full = smem_at(&st.q_full), q_empty = smem_at(&st.q_empty), k_full = smem_at(st.k_full),
                 k_empty = smem_at(st.k_empty), v_full = smem_at(st.v_full), v_empty = smem_at(st.v_empty),
                 s_full = smem_at(&st.s_full), s_empty = smem_at(&st.s_empty), dp_full = smem_at(st.dp_full),
                 ds_full = smem_at(st.ds_full), done = smem_at(&st.done), clean = smem_at(st.clean), scored_at = smem_at(st.scored);
  const Dead dead = {&st.dead, a.polls};
  if (threadIdx.x == 0) {
    st.dead = st.bad = 0;
#pragma unroll 1
    for (int i = 0; i < kKeyStages; ++i) {
      mbar_init(clean + 8 * i, 1);
      mbar_init(scored_at + 8 * i, 1);
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 2);  // the matrix instructions and the cleaning warp
    }
#pragma unroll 1
    for (int i = 0; i < kValueStages; ++i) {
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(s_empty, 8);
    mbar_init(dp_full, 1);
    mbar_init(dp_full + 8, 1);
    mbar_init(done, 1);
    for (int i = 0; i < 4; ++i) mbar_init(ds_full + 8 * i, 4);
    init_work(st.work, 11);  // eight warps of the arithmetic, copies, cleaning, matrix instructions
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
  auto take = [&](int k) { return take_work(st.work, st.item, k, lane, dead); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 11) {  // ---- work
      find_work(st.work, st.item, blockIdx.x, false, lane, dead, [&](uint32_t id) {
        fill_rest(a.cu_q, a.nseq, a.num_q, (int64_t)a.heads * a.d / 8, static_cast<uint4*>(a.dq), (int64_t)id * 32 + lane,
                  (int64_t)gridDim.x * 32);
        return rows_item(a, id, gridDim.x, lane);
      });
    } else if (warp == 9) {  // ---- copies
      Place<kKeyStages> at = {0, 0};
      Place<kValueStages> value = {0, 0};
      uint32_t loaded = 0, k_tiles = 0, v_tiles = 0;
#pragma unroll 1
      for (int k = 0;; ++k) {
        const RowsItem x = take(k);
        if (x.n0 < 0) break;
        if (x.n0 == 0) continue;
        if (lane == 0) wait_for(q_empty, (loaded & 1) ^ 1, dead);
        if (lane == 0 && !*dead) {
          ++loaded;
          mbar_expect(q_full, 2 * (C::DP / 64) * 128 * rows);
          load_tile<C>(q_at, &mq, x.kvh * a.group, x.w.q0 + x.t0, q_full);
          load_tile<C>(g_at, &mg, x.kvh * a.group, x.w.q0 + x.t0, q_full);
#pragma unroll 1
          for (int j = 0; j < x.n0; ++j) {
            wait_for(k_empty + 8 * at.stage, at.parity ^ 1, dead);
            if (*dead) break;
            ++k_tiles;
            mbar_expect(k_full + 8 * at.stage, C::TILE);
            load_tile<C>(k_at + at.stage * C::TILE, &mk, x.kvh, x.w.k0 + (x.kb0 + j) * 128, k_full + 8 * at.stage);
            at.next(1);
            wait_for(v_empty + 8 * value.stage, value.parity ^ 1, dead);
            if (*dead) break;
            ++v_tiles;
            mbar_expect(v_full + 8 * value.stage, C::TILE);
            load_tile<C>(v_at + value.stage * C::TILE, &mv, x.kvh, x.w.k0 + (x.kb0 + j) * 128, v_full + 8 * value.stage);
            value.next(1);
          }
        }
        __syncwarp();
      }
      if (lane == 0) {
        land_ring(q_full, 1, loaded);
        land_ring(k_full, kKeyStages, k_tiles);
        land_ring(v_full, kValueStages, v_tiles);
      }
    } else if (warp == 10) {  // ---- infinities and NaN of keys that not every row sees
      // S is formed from them as they are (a key may hold -inf to have no weight), so it comes first.
      Place<kKeyStages> at = {0, 0};
      uint32_t cleaned = 0;  // a parity a stage
#pragma unroll 1
      for (int k = 0;; ++k) {
        const RowsItem x = take(k);
        if (x.n0 < 0) break;
#pragma unroll 1
        for (int j = 0; j < x.n0; ++j) {
          // every block is waited for, and its place held until this warp has seen it: a parity
          // tells only whether the one before it in its place has come
          wait_for(k_full + 8 * at.stage, at.parity, dead);
          if (rows_mixed(a, x, j)) {
            wait_for(scored_at + 8 * at.stage, (cleaned >> at.stage) & 1, dead);
            cleaned ^= 1u << at.stage;
            clean_operand<C::HALF>(k_ptr + at.stage * C::TILE, C::TILE, lane, &st.bad);
            __syncwarp();
            if (lane == 0) mbar_arrive(clean + 8 * at.stage);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(k_empty + 8 * at.stage);
          tile_seen(st.work, lane);
          at.next(1);
        }
      }
    } else if (warp == 8) {  // ---- matrix instructions
      const uint32_t leader = tc_leader(), tm = uniform(tmem), S = tm, DP = tm + 128, DQ = tm + 384;
      Place<kKeyStages> key = {0, 0}, used = {0, 0};  // of the next S, of the next dQ
      Place<kValueStages> value = {0, 0};
      uint32_t scored = 0, weighed = 0, added = 0, items = 0, cleaned = 0;  // cleaned: a parity a stage
      auto scores = [&](bool mixed) {
        wait_for(k_full + 8 * key.stage, key.parity, dead);
        wait_for(s_empty, (scored & 1) ^ 1, dead);
        tc_after();
        product<C>(leader, S, q_at, k_at + key.stage * C::TILE);
        tc_commit_by(leader, s_full);
        if (mixed) tc_commit_by(leader, scored_at + 8 * key.stage);
        ++scored;
        key.next(1);
      };
      auto weights = [&]() {  // dP
        wait_for(v_full + 8 * value.stage, value.parity, dead);
        tc_after();
        product<C>(leader, DP + 128 * (weighed & 1), g_at, v_at + value.stage * C::TILE);
        tc_commit_by(leader, v_empty + 8 * value.stage);
        tc_commit_by(leader, dp_full + 8 * (weighed & 1));
        ++weighed;
        value.next(1);
      };
#pragma unroll 1
      for (int k = 0;; ++k) {
        const RowsItem x = take(k);
        const int n = (int)uniform((uint32_t)x.n0);
        if (n < 0) break;
        if (n == 0) continue;
        wait_for(q_full, items & 1, dead);
        ++items;
        const int2 whole = rows_whole(a, x);
        const int from = (int)uniform((uint32_t)whole.x), to = (int)uniform((uint32_t)whole.y);
        auto mixed = [&](int j) { return j < from || j >= to; };
        scores(mixed(0));
        weights();
        if (n > 1) {
          weights();
          scores(mixed(1));
        }
        if (n <= 2) tc_commit_by(leader, q_empty);
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          if (j == max(0, n - 3)) want_work(st.work, lane);
          const uint32_t ready = ds_full + 16 * (added & 1), parity = (added >> 1) & 1;
          if (mixed(j)) {
            wait_for(clean + 8 * used.stage, (cleaned >> used.stage) & 1, dead);
            cleaned ^= 1u << used.stage;
          }
          // the item's first product writes over sums that both groups have to have read
          if (j == 0) wait_for(ready + 8, parity, dead);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            wait_for(ready + 8 * half, parity, dead);
            tc_after();
            product_add<C>(leader, DQ, DP + 128 * (added & 1), k_at + used.stage * C::TILE, half, j > 0 || half > 0);
          }
          ++added;
          tc_commit_by(leader, k_empty + 8 * used.stage);
          used.next(1);
          if (j + 2 < n) {
            weights();
            scores(mixed(j + 2));
            if (j + 3 == n) tc_commit_by(leader, q_empty);
          }
        }
        tc_commit_by(leader, done);
      }
      end_products(st.work, leader);
    }
  } else {  // ---- dS: a row a thread, half of a block's keys
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MATH_REGS));
    const int half = warp >> 2, col = half * 64, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int in_tile = r / a.group, head = r - in_tile * a.group, e = gradient_exponent<C::HALF>(b);
    RowsMath m = {dead, tmem + lanes + col, tmem + 128 + lanes + col, s_full, s_empty, dp_full, ds_full + 8 * half, 0, 0, false,
                  a.scale * kLog2e, C::HALF ? exp2f((float)-e) : 1.0f, 0.0f, 0.0f};
    uint32_t tiles = 0, items = 0;
#pragma unroll 1
    for (int k = 0;; ++k) {
      const RowsItem x = take(k);
      if (x.n0 < 0) break;
      const int token = x.t0 + in_tile;
      const bool there = r < rows && token < x.t1;
      const int64_t row = (int64_t)(x.w.q0 + token) * a.heads + x.kvh * a.group + head;
      const float2 stats = there ? __ldg(b.stats + row) : make_float2(-INFINITY, 0.0f);
      const int hi = there ? x.off + token + 1 : 0, lo = a.window ? max(0, hi - a.window) : 0;
      m.hi = hi - x.kb0 * 128 - col;
      m.lo = lo - x.kb0 * 128 - col;
      m.single = hi - lo == 1;
      m.lse = stats.x;
      m.delta = stats.y * m.f;
#pragma unroll 1
      for (int j = 0; j < x.n0; ++j, ++tiles) {
        if (rows_mixed(a, x, j))
          rows_step_some<C>(m, tiles, j * 128);
        else
          rows_step<C, false>(m, tiles, 0);
      }
      if (x.n0 > 0) wait_for(done, items++ & 1, dead);
      tc_after();
      float factor = a.scale * (C::HALF ? exp2f((float)(e - 15)) : 1.0f);
      if (*dead) factor = NAN;
#pragma unroll 1
      for (int i = half * (C::DP / 2); i < (half + 1) * (C::DP / 2); i += 32) {
        float o[32];
        if (x.n0 > 0) tc_load32(tmem + 384 + lanes + i, o);
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = x.n0 > 0 ? o[c] * factor : 0.0f;
        if (there && i < a.d) store_columns<C::HALF>(a.dq, row * a.d, a.d, i, o);
      }
      tc_before();
    }
  }
  __syncwarp();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (*dead)
    for_last_items(st.work, [&](uint32_t id) {
      const RowsItem x = rows_item(a, id, gridDim.x, lane);
      const int vectors = a.d / 8;
#pragma unroll 1
      for (int i = threadIdx.x; i < (x.t1 - x.t0) * a.group * vectors; i += C::THREADS) {
        const int r = i / vectors;
        const int64_t row = (int64_t)(x.w.q0 + x.t0 + r / a.group) * a.heads + x.kvh * a.group + r % a.group;
        put_nan(a.dq, row, vectors, i % vectors);
      }
    });
}

template <class C>
cudaError_t launch_passes(const BwdArgs& b, cudaStream_t stream) {
  const PromptArgs& a = b.a;
  constexpr int KEYS_SMEM = 1024 + C::HEAD + 6 * C::TILE, ROWS_SMEM = 2048 + (2 + kKeyStages + kValueStages) * C::TILE;
  const int tp = 128 / a.group;
  CUtensorMap mq, mk, mv, mg;
  cudaError_t e = rows_map(&mq, a.q, C::HALF, a.d, a.heads, a.num_q, a.qt, a.qh, a.group, tp);
  if (e == cudaSuccess) e = rows_map(&mg, a.g, C::HALF, a.d, a.heads, a.num_q, a.gt, a.gh, a.group, tp);
  if (e == cudaSuccess) e = rows_map(&mk, a.k, C::HALF, a.d, a.kv, a.num_k, a.kt, a.kh, 1, 128);
  if (e == cudaSuccess) e = rows_map(&mv, a.v, C::HALF, a.d, a.kv, a.num_k, a.vt, a.vh, 1, 128);
  auto* keys = prompt_keys_kernel<C>;
  auto* rows = prompt_rows_kernel<C>;
  if (e == cudaSuccess) e = allow_dynamic_smem((const void*)keys, KEYS_SMEM);
  if (e == cudaSuccess) e = allow_dynamic_smem((const void*)rows, ROWS_SMEM);
  if (e != cudaSuccess) return e;
  if (a.num_k > 0) {
    const int64_t blocks = ((int64_t)a.num_k / 128 + a.nseq) * a.kv;
    e = launch_dependent(keys, dim3((unsigned)blocks), dim3(C::THREADS), KEYS_SMEM, stream, b, mq, mk, mv, mg);
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks = ((int64_t)a.num_q / tp + a.nseq) * a.kv;
  return launch_dependent(rows, dim3((unsigned)blocks), dim3(C::THREADS), ROWS_SMEM, stream, b, mq, mk, mv, mg);
}

}  // namespace

cudaError_t launch_prompt_bwd(const PromptArgs& a, bool half, cudaStream_t stream) {
  BwdArgs b = {};
  b.a = a;
  const int tp = 128 / a.group;
  // one CTA an SM resides, by its registers
  const bool many = (a.window ? std::min((int64_t)a.num_q, (int64_t)a.window + 128) : a.num_q) / tp + 1 > kSumTiles;
  b.places = many ? sm_count() : 0;
  const size_t stats = sizeof(float2) * (size_t)a.num_q * a.heads, place = sizeof(float) * 2 * 128 * (a.d <= 64 ? 64 : 128),
               flags = 16 + sizeof(uint32_t) * (size_t)b.places;
  void* ws = nullptr;
  cudaError_t e = workspace_take(&ws, place * b.places + stats + flags, stream);
  if (e != cudaSuccess) return e;
  if (many) b.sums = static_cast<float*>(ws);
  b.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + place * b.places);
  b.sizes = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(b.stats) + stats);
  b.taken = b.sizes + 4;
  if (half || many) e = cudaMemsetAsync(b.sizes, 0, flags, stream);
  if (e == cudaSuccess) {
    const int64_t most = half && a.num_k > a.num_q ? a.num_k : a.num_q;
    int64_t blocks = (most + 3) / 4;
    if (blocks > 152 * 16) blocks = 152 * 16;
    e = half ? launch_dependent(prompt_delta_kernel<true>, dim3((unsigned)blocks), dim3(128), 0, stream, b)
             : launch_dependent(prompt_delta_kernel<false>, dim3((unsigned)blocks), dim3(128), 0, stream, b);
  }
  if (e == cudaSuccess) {
    if (a.d <= 64)
      e = half ? launch_passes<Bwd<64, true>>(b, stream) : launch_passes<Bwd<64, false>>(b, stream);
    else
      e = half ? launch_passes<Bwd<128, true>>(b, stream) : launch_passes<Bwd<128, false>>(b, stream);
  }
  const cudaError_t ef = workspace_give(ws, stream);
  return e != cudaSuccess ? e : ef;
}

}  // namespace csa
