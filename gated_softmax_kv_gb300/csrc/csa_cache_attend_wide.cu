// Attention over the 8-bit cache for many query rows of one cache head (large
// groups of heads, chunks of a prompt): tcgen05.
//
// One CTA an SM works on a tile of R = 64 query rows and runs over the keys 128
// at a time, transposed so that the accumulator's lanes are keys, then columns:
//   S^T [128 keys x R] = K [128 x D] Q^T        (TMEM, two buffers)
//   O^T [D x R] += V^T [D x 128] P^T            (TMEM, D / 128 tiles of 128 x R)
// Heads of 64 columns fill half a panel; the other half holds them again.
// TMEM's 512 columns hold 2 R + R D / 128 of them. The rows are the N of both
// products, so 64 heads fill the tensor core as well as 128 do.
//
// Roles: producer warps read the 8-bit rows into registers several panels
// ahead, widen them to fp16 (exact) and store them to a ring of panels (128 keys
// x 128 columns) in shared memory in the 128-byte swizzle; a panel is the
// K-major operand of S^T and, unchanged, the M-major operand of O^T, so a row
// that is key and value is stored once. A warp of its own issues the matrix
// instructions. Softmax warps own a key a thread: they read S^T from TMEM, form
// the weights and store P^T [key][row], the N-major operand.
//
// Numerics as in csa_cache_attend_rows.cu: references m and m' that rise only
// when passed, fp16 weights that carry the value scale. Where scales lie
// within 2^30 and the references within 2^60 of one another, the weight is the
// softmax term times two factors; beyond, it takes an exponential of its own.
//
// What bounds it: shared memory and the chain. A tile of 128 keys of 512 columns
// costs 64 instructions of 128 x 64 x 16 (3.1 K cycles at 6 KB of operands and
// 128 bytes a cycle each), 128 KB of stores (1 K) and the softmax (2.4 K); heads
// of 512 have room for one tile in the ring, so refill, S^T, softmax and O^T
// follow one another: 8.8 K cycles a tile. Seven producer warps measured best (six
// 201 us, eight 238, seven 192). Measured: 64 sequences of 10400 rows on average,
// 64 heads over one row of 512: 188 us (451 TFLOP/s), joining 14 us; one sequence
// of 65536 rows 44 us, joining 8; 255 queries each of four sequences of up to 4099 rows, 16
// heads over two of 128 columns, 82 us, joining 8; 2048 queries of 64 heads over 4096
// rows of 512, 2061 us (500 TFLOP/s).
//
// Every wait on an mbarrier is bounded: a wait that runs out marks the CTA,
// whose later waits then return at once, and its results become NaN.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache_attend.h"
#include "csa_cache_join.cuh"
#include "csa_cache_plan.cuh"
#include "csa_device.cuh"
#include "csa_e4m3.cuh"
#include "csa_tc.cuh"

namespace csa {

namespace {

// One item of work, as the roles read it.
struct WideItem {
  const uint8_t* data;
  const float* scales;
  const int32_t* row_table;  // the sequence's row of the page table
  float* ws;                 // slot for a partial result
  uint16_t* out;
  float* lse;
  int64_t c0;                // first tile of 128 keys
  int32_t n;                 // tiles of 128 keys
  int32_t least, most;       // rows that the queries see: fewest, most
  int32_t key_head, value_head, heads, num_pages, page_bits, block_bits;
  uint32_t panels_done, tiles_done;  // of earlier items: ring slots and barrier phases
  bool whole;                // from the item's first key to its last
};

// Shared memory in front of the ring. The roles are functions of their own, so
// that each has the registers to itself; they reach it through wide_smem.
template <int R, int NS, int WARPS>
struct WideState {
  // read four at a time; see wide_softmax
  alignas(16) float zf[R];
  alignas(16) float mref[R];
  alignas(16) float mpref[R];
  alignas(16) float rl[R];
  alignas(16) float rf[R];
  alignas(16) int32_t sees[R];
  alignas(16) int64_t sums[WARPS + 1];
  int64_t row_at[R], q_at[R];
  uint64_t bars[2 * NS + 6];
  Place found;
  WideItem item;
  float lscale[R], oscale[R], factor[R];
  float best[2][R / 32][4][32];
  float part[R * 4];
  // Whether a row's references are too far apart for weights in two factors: one
  // of each half of the rows, written and read by that half's four warps alone,
  // which their own barrier orders.
  int32_t far_refs[R / 32];
  int32_t sees_least, sees_most, nan_rows, dead, first_nan;
  uint32_t tmem;
};
extern __shared__ __align__(1024) uint8_t wide_smem[];

template <int D, bool SHARED>
struct Wide {
  static constexpr int R = 64;                      // query rows of a tile
  static constexpr int PP = (D + 127) / 128;        // panels of 128 keys; of D = 64 the columns come twice
  static constexpr int SW = R / 8;                  // softmax warps: 4 for each 32 rows
  static constexpr int PW = 7;                      // producer warps
  static constexpr int THREADS = (SW + PW + 1) * 32;  // 16 warps: 128 registers a thread
  static constexpr int NS = 4;                      // panels of the ring
  static constexpr bool AHEAD = !SHARED || 2 * PP <= NS;  // S^T of the next keys before O^T of these
  static constexpr int SLAB = 16384;                // 128 keys x 64 columns
  static constexpr int PANEL = 2 * SLAB;
  static constexpr int QSLAB = R * 128;
  static constexpr int Q = R * D * 2;
  static constexpr int P = R * 256;                 // [128 keys][R rows]: one 128-byte line a key
  static_assert(R == 64, "a line of P^T holds 64 rows");
  using State = WideState<R, NS, THREADS / 32>;
  static constexpr int HEAD = (int)(sizeof(State) + 1023) / 1024 * 1024;
  static constexpr int SMEM = HEAD + NS * PANEL + Q + P + 1024;
  static constexpr int KV = (32 + PW - 1) / PW;     // steps of 4 keys a warp and panel
  // Step k of producer warp pw is keys 4 e .. 4 e + 3 of the tile, e = step_of(k, pw).
  // The warps for which a last step would be one too many repeat their own before
  // it, so that no two warps ever store, or clean, the same keys.
  static __host__ __device__ constexpr int step_of(int k, int pw) {
    return k * PW + pw < 32 ? k * PW + pw : (k - 1) * PW + pw;
  }
  static constexpr bool each_step_by_one_warp() {
    int owner[32] = {}, steps = 0;
    for (int pw = 0; pw < PW; ++pw)
      for (int k = 0; k < KV; ++k) {
        const int e = step_of(k, pw);
        if (e < 0 || e >= 32 || (owner[e] != 0 && owner[e] != pw + 1)) return false;
        steps += owner[e] == 0;
        owner[e] = pw + 1;
      }
    return steps == 32;
  }
  // Panels in flight in registers. Heads of one panel (128 columns) have less to
  // wait for and the lookups in every panel: one measured 82 us, two 87 (1020
  // queries of 16 heads over 16396 rows); of four panels two measured less.
  static constexpr int DEPTH = PP == 1 ? 1 : 2;
  static constexpr int SLOT = R * (D + 4);
  static constexpr uint32_t S0 = 0, O0 = 2 * R;     // TMEM columns
  // fp32 accumulator, fp16 operands, N = R, M = 128; O^T has both transposed.
  static constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(R >> 3) << 17) | (8u << 24);
  static constexpr uint32_t IDESC_O = IDESC_S | (1u << 15) | (1u << 16);
};

// Where everything is, from the role's point of view.
template <class C>
struct Places {
  uint32_t ring, q, p, full, empty, s_full, s_empty, p_full, p_empty;
  uint8_t* ring_ptr;
};
template <class C>
__device__ __forceinline__ Places<C> places() {
  Places<C> x;
  const uint32_t base = smem_at(wide_smem);
  x.ring = (base + C::HEAD + 1023u) & ~1023u;
  x.ring_ptr = wide_smem + (x.ring - base);
  x.q = x.ring + C::NS * C::PANEL;
  x.p = x.q + C::Q;
  x.full = smem_at(reinterpret_cast<typename C::State*>(wide_smem)->bars);
  x.empty = x.full + 8 * C::NS;
  x.s_full = x.empty + 8 * C::NS;
  x.s_empty = x.s_full + 16;
  x.p_full = x.s_empty + 16;
  x.p_empty = x.p_full + 8;
  return x;
}

// Largest over the warp of each of 32 values: lane i gets that of v[i].
__device__ __forceinline__ float column_max(float* v, int lane) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float keep = lane & o ? v[j + o] : v[j], send = lane & o ? v[j] : v[j + o];
      v[j] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
    }
  return v[0];
}

// Which rows the tile has, what each sees, where it is written: a thread a row.
template <int D, bool SHARED>
__device__ __forceinline__ void stage_rows(const AttendArgs& a, int s, int64_t tile, int h, int64_t keys) {
  using C = Wide<D, SHARED>;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  const int i = threadIdx.x;
  if (i >= C::R) return;
  const Row w = row_of(a, s, tile, h, C::R, i);
  int32_t limit = 0x7FFFFFFF;
  if (w.there && a.visible) limit = __ldg(a.visible + w.token);
  const int sees = (int)min(keys, (int64_t)max(limit, 0));
  st.sees[i] = w.there ? sees : 0x7FFFFFFF;  // rows that are not there are not looked at
  st.row_at[i] = w.there ? w.token * a.heads + w.head : -1;
  st.q_at[i] = w.there ? w.token * a.qt + w.head * a.qh : -1;
  st.mref[i] = st.mpref[i] = kNone;
  st.rl[i] = kLift;
  st.rf[i] = 128.0f;
  const int lo = __reduce_min_sync(0xFFFFFFFFu, w.there ? sees : 0x7FFFFFFF);
  const int hi = __reduce_max_sync(0xFFFFFFFFu, w.there ? sees : 0);
  if ((i & 31) == 0) {
    atomicMin(&st.sees_least, lo);
    atomicMax(&st.sees_most, hi);
  }
}

// Q's rows as fp16 in the K-major operand's layout, scaled row by row, by the
// softmax warps.
template <int D, bool SHARED, bool HALF>
__device__ __forceinline__ void stage_queries(const uint16_t* q, float scale) {
  using C = Wide<D, SHARED>;
  constexpr int R = C::R, EACH = R / C::SW;
  constexpr int V = D / 256 > 0 ? D / 256 : 1;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  uint8_t* to = places<C>().ring_ptr + C::NS * C::PANEL;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4 x[EACH][V];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {  // all loads first
    const int64_t at = st.q_at[warp + e * C::SW];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (k * 32 + lane) * 8;
      x[e][k] = at >= 0 && col < D ? __ldg(reinterpret_cast<const uint4*>(q + at + col))
                                   : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int i = warp + e * C::SW;
    const int lift = query_lift<HALF>(finite_max<HALF, V>(x[e]));
    const float f = exp2i(lift);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (k * 32 + lane) * 8;
      if (col < D)
        *reinterpret_cast<uint4*>(to + (col >> 6) * C::QSLAB + i * 128 + ((((col >> 3) & 7) ^ (i & 7)) << 4)) =
            lifted<HALF>(x[e][k], f);
    }
    if (lane == 0) st.zf[i] = scale * exp2i(-lift);
  }
}

// The order of the planes. A plane is one tile of keys or of values (or,
// shared, of both): PP panels. They are loaded, and used by the matrix
// instructions, as K0, K1, V0, K2, V1, ...
template <bool SHARED>
struct Planes {
  int n;  // tiles
  __device__ __forceinline__ int count() const { return SHARED ? n : 2 * n; }
  __device__ __forceinline__ int tile(int q) const {
    if (SHARED) return q;
    if (q == 2 * n - 1) return n - 1;
    return q == 0 ? 0 : (q & 1) ? (q + 1) / 2 : q / 2 - 1;
  }
  __device__ __forceinline__ bool value(int q) const {
    return !SHARED && q > 0 && (q == 2 * n - 1 || (q & 1) == 0);
  }
  __device__ __forceinline__ int keys_of(int i) const { return SHARED ? i : i == 0 ? 0 : 2 * i - 1; }
  __device__ __forceinline__ int values_of(int i) const {
    return SHARED ? i : i == n - 1 ? 2 * n - 1 : 2 * i + 2;
  }
};

// The matrix instructions, issued by a warp of their own (all of its lanes call
// these, one is elected). The operands' descriptors differ by constants, which
// keeps the issue ahead of the tensor core: 48 cycles an instruction of 128 x
// 64 x 16, set by the 6 KB of operands that it reads from shared memory.
template <int D, bool SHARED>
struct Issue {
  using C = Wide<D, SHARED>;
  const Places<C>& at;
  Planes<SHARED> planes;
  volatile int32_t* dead;
  uint32_t tmem, panels_done, tiles_done;

  __device__ __forceinline__ void scores(int i) const {  // S^T of tile i
    const uint32_t tc = tiles_done + i, b = tc & 1;
    mbar_wait(at.s_empty + 8 * b, ((tc >> 1) & 1) ^ 1, dead);
    for (int pp = 0; pp < C::PP; ++pp) {
      const uint32_t pc = panels_done + planes.keys_of(i) * C::PP + pp, slot = pc % C::NS;
      mbar_wait(at.full + 8 * slot, (pc / C::NS) & 1, dead);
      tc_after();
      __syncwarp();
      const uint64_t k = operand(at.ring + slot * C::PANEL, 16);
      const uint64_t q = operand(at.q + pp * 2 * C::QSLAB, 16);
#pragma unroll
      for (int j = 0; j < (D < 128 ? 4 : 8); ++j)
        tc_mma(tmem + C::S0 + b * C::R, k + ((j >> 2) * C::SLAB + (j & 3) * 32) / 16,
               q + ((j >> 2) * C::QSLAB + (j & 3) * 32) / 16, C::IDESC_S, pp > 0 || j > 0);
      if (!SHARED) tc_commit(at.empty + 8 * slot);
    }
    tc_commit(at.s_full + 8 * b);
  }
  __device__ __forceinline__ void values(int i) const {  // O^T += V^T P^T of tile i
    const uint32_t tc = tiles_done + i;
    mbar_wait(at.p_full, tc & 1, dead);
    tc_after();
    const uint64_t p = operand(at.p, 1024);
    for (int pp = 0; pp < C::PP; ++pp) {
      const uint32_t pc = panels_done + planes.values_of(i) * C::PP + pp, slot = pc % C::NS;
      if (!SHARED) {
        mbar_wait(at.full + 8 * slot, (pc / C::NS) & 1, dead);
        tc_after();
      }
      __syncwarp();
      const uint64_t v = operand(at.ring + slot * C::PANEL, C::SLAB);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        tc_mma(tmem + C::O0 + pp * C::R, v + j * 128, p + j * 128, C::IDESC_O, i > 0 || j > 0);
      tc_commit(at.empty + 8 * slot);
    }
    tc_commit(at.p_empty);
  }
};

template <int D, bool SHARED>
__device__ __noinline__ void wide_products() {
  using C = Wide<D, SHARED>;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  const Places<C> at = places<C>();
  const int n = (int)uniform((uint32_t)st.item.n);
  const Issue<D, SHARED> issue = {at, {n}, &st.dead, uniform(st.tmem), uniform(st.item.panels_done),
                                  uniform(st.item.tiles_done)};
  if (C::AHEAD && n > 0) issue.scores(0);
  for (int i = 0; i < n; ++i) {
    if (!C::AHEAD)
      issue.scores(i);
    else if (i + 1 < n)
      issue.scores(i + 1);
    issue.values(i);
  }
}

// Some weight passes its reference: both references rise to the tile's maxima,
// and what O^T has so far is scaled down. By the four warps of 32 rows; each
// thread has a key, as in wide_softmax, which scales its sums by lscale.
template <int D, bool SHARED>
__device__ __noinline__ void wide_raise(uint32_t s_at, float sk, float lv, bool there, int64_t key, uint32_t tc,
                                        int i) {
  using C = Wide<D, SHARED>;
  constexpr int R = C::R;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quarter = warp & 3, half = warp >> 2, col = half * 32;
  float t[32];
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {  // z, then z + log2(value scale)
    tc_load32(s_at, t);
    const float add = k ? lv : 0.0f;
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 z4 = *reinterpret_cast<const float4*>(st.zf + col + c);
      const int4 n4 = *reinterpret_cast<const int4*>(st.sees + col + c);
      t[c] = there && key < n4.x ? __fmul_rn(t[c], __fmul_rn(sk, z4.x)) + add : -INFINITY;
      t[c + 1] = there && key < n4.y ? __fmul_rn(t[c + 1], __fmul_rn(sk, z4.y)) + add : -INFINITY;
      t[c + 2] = there && key < n4.z ? __fmul_rn(t[c + 2], __fmul_rn(sk, z4.z)) + add : -INFINITY;
      t[c + 3] = there && key < n4.w ? __fmul_rn(t[c + 3], __fmul_rn(sk, z4.w)) + add : -INFINITY;
    }
    st.best[k][half][quarter][lane] = column_max(t, lane);
  }
  if (tc > 0) mbar_wait(places<C>().p_empty, (tc - 1) & 1, &st.dead);
  tc_after();
  barrier_of(1 + half, 128);
  if (quarter == 0) {
    const int c = col + lane;
    float x = st.mref[c], y = st.mpref[c];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x = fmaxf(x, st.best[0][half][k][lane]);
      y = fmaxf(y, st.best[1][half][k][lane]);
    }
    st.lscale[c] = exp2f(st.mref[c] - x);
    st.oscale[c] = exp2f(st.mpref[c] - y);
    st.mref[c] = x;
    st.mpref[c] = y;
    st.rl[c] = x - y + kLift;
    st.rf[c] = exp2f(x - y + kLift);
    if (!(fabsf(x - y) <= 60.0f)) st.far_refs[half] = 1;
  }
  barrier_of(1 + half, 128);
  if (i > 0) {
#pragma unroll 1
    for (int pp = 0; pp < C::PP; ++pp) {
      const uint32_t o_at = st.tmem + ((uint32_t)(quarter * 32) << 16) + C::O0 + pp * R + col;
      tc_load32(o_at, t);
#pragma unroll
      for (int c = 0; c < 32; ++c) t[c] *= st.oscale[col + c];
      tc_store32(o_at, t);
    }
  }
}

// The softmax warps. A thread has key `mine` of each tile and 32 of the rows.
// For a row: z = S * (key scale * zf) in log2 units, t = z - mref; the weight is
// 2^(t + log2(value scale) + rl), rl = mref - mpref + 7, rf = 2^rl.
template <int D, bool SHARED>
__device__ __noinline__ void wide_softmax() {
  using C = Wide<D, SHARED>;
  constexpr int R = C::R;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  const Places<C> at = places<C>();
  const WideItem& item = st.item;
  volatile int32_t* dead = &st.dead;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c0 = item.c0;
  const int n = item.n, least = item.least, most = item.most;
  const uint32_t tmem = st.tmem, tiles_done = item.tiles_done;
  const int quarter = warp & 3, half = warp >> 2, mine = quarter * 32 + lane;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const int col = half * 32;
  uint8_t* p_line = at.ring_ptr + C::NS * C::PANEL + C::Q + mine * 128;
  float l[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) l[c] = 0.0f;
  auto page_at = [&](int i) -> int32_t {
    const int64_t key = (c0 + i) * 128 + mine;
    return i < n && key < most ? __ldg(item.row_table + (key >> item.page_bits)) : -1;
  };
  float sk_next, sv_next;
  auto scales_at = [&](int i, int32_t page) {  // of this thread's key of tile i; -1: no row
    sk_next = -1.0f;
    sv_next = 1.0f;
    if (page >= 0 && page < item.num_pages) {
      const int slot = (int)(((c0 + i) * 128 + mine) & ((1 << item.page_bits) - 1));
      const int64_t first = (int64_t)page * item.heads;
      const int bits = item.page_bits - item.block_bits;
      const float* block = item.scales + (slot >> item.block_bits);
      sk_next = __ldg(block + ((first + item.key_head) << bits));
      sv_next = SHARED ? sk_next : __ldg(block + ((first + item.value_head) << bits));
    }
  };
  scales_at(0, page_at(0));
  int32_t page_next = page_at(1);
  for (int i = 0; i < n; ++i) {
    const uint32_t tc = tiles_done + i, b = tc & 1;
    const float sk = sk_next;
    const bool there = !(sk < 0.0f);
    const float lv = there ? __log2f(sv_next) : 0.0f;
    const float kf = ex2_approx_ftz(lv);
    scales_at(i + 1, page_next);
    page_next = page_at(i + 2);
    const int64_t key = (c0 + i) * 128 + mine;
    // some row does not see some key of the tile, or a page is missing
    const bool mixed = (c0 + i + 1) * 128 > least || !there;
    const bool far_key = !(fabsf(lv) <= 30.0f);
    mbar_wait(at.s_full + 8 * b, (tc >> 1) & 1, dead);
    tc_after();
    const uint32_t s_at = tmem + lanes + C::S0 + b * R + col;
    const float2 sk2 = make_float2(sk, sk), lv2 = make_float2(lv, lv);
    float t[32];
    bool o_free = false;  // O^T of the tile before is complete
    for (int attempt = 0;; ++attempt) {
      if (i == 0 && attempt == 0) {  // there is no reference yet; the sums are 0
        wide_raise<D, SHARED>(s_at, sk, lv, there, key, tc, i);
        o_free = true;
        continue;
      }
      tc_load32(s_at, t);
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 z4 = *reinterpret_cast<const float4*>(st.zf + col + c);
        const float4 m4 = *reinterpret_cast<const float4*>(st.mref + col + c);
        const float2 ca = mul2_rn(make_float2(z4.x, z4.y), sk2);
        const float2 cb = mul2_rn(make_float2(z4.z, z4.w), sk2);
        const float2 ta = sub2_rn(make_float2(__fmul_rn(t[c], ca.x), __fmul_rn(t[c + 1], ca.y)),
                                  make_float2(m4.x, m4.y));
        const float2 tb = sub2_rn(make_float2(__fmul_rn(t[c + 2], cb.x), __fmul_rn(t[c + 3], cb.y)),
                                  make_float2(m4.z, m4.w));
        t[c] = ta.x;
        t[c + 1] = ta.y;
        t[c + 2] = tb.x;
        t[c + 3] = tb.y;
      }
      if (mixed) {  // rows that do not see this key
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const int4 n4 = *reinterpret_cast<const int4*>(st.sees + col + c);
          t[c] = there && key < n4.x ? t[c] : -INFINITY;
          t[c + 1] = there && key < n4.y ? t[c + 1] : -INFINITY;
          t[c + 2] = there && key < n4.z ? t[c + 2] : -INFINITY;
          t[c + 3] = there && key < n4.w ? t[c + 3] : -INFINITY;
        }
      }
      float mx = -INFINITY, mw = -INFINITY;
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 r4 = *reinterpret_cast<const float4*>(st.rl + col + c);
        const float2 wa = add2_rn(make_float2(t[c], t[c + 1]), add2_rn(make_float2(r4.x, r4.y), lv2));
        const float2 wb = add2_rn(make_float2(t[c + 2], t[c + 3]), add2_rn(make_float2(r4.z, r4.w), lv2));
        mx = fmaxf(fmaxf(mx, t[c]), fmaxf(t[c + 1], fmaxf(t[c + 2], t[c + 3])));
        mw = fmaxf(fmaxf(mw, wa.x), fmaxf(wa.y, fmaxf(wb.x, wb.y)));
      }
      if (attempt > 0 || !barrier_any(1 + half, 128, mx > kSlackM || mw > kSlackW + kLift)) break;
      wide_raise<D, SHARED>(s_at, sk, lv, there, key, tc, i);
      o_free = true;
#pragma unroll
      for (int c = 0; c < 32; ++c) l[c] *= st.lscale[col + c];
    }
    tc_before();  // S^T is read
    __syncwarp();
    if (lane == 0) mbar_arrive(at.s_empty + 8 * b);
    const bool far = __any_sync(0xFFFFFFFFu, far_key) || *(volatile int32_t*)&st.far_refs[half];
    uint32_t w[16];
    if (!far) {
      const float2 kf2 = make_float2(kf, kf);
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 f4 = *reinterpret_cast<const float4*>(st.rf + col + c);
        const float2 pa = make_float2(ex2_approx_ftz(t[c]), ex2_approx_ftz(t[c + 1]));
        const float2 pb = make_float2(ex2_approx_ftz(t[c + 2]), ex2_approx_ftz(t[c + 3]));
        const float2 la = add2_rn(make_float2(l[c], l[c + 1]), pa);
        const float2 lb = add2_rn(make_float2(l[c + 2], l[c + 3]), pb);
        l[c] = la.x;
        l[c + 1] = la.y;
        l[c + 2] = lb.x;
        l[c + 3] = lb.y;
        const float2 wa = mul2_rn(pa, mul2_rn(make_float2(f4.x, f4.y), kf2));
        const float2 wb = mul2_rn(pb, mul2_rn(make_float2(f4.z, f4.w), kf2));
        w[c / 2] = pack_f16x2(wa.x, wa.y);
        w[c / 2 + 1] = pack_f16x2(wb.x, wb.y);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        l[c] += ex2_approx_ftz(t[c]);
        l[c + 1] += ex2_approx_ftz(t[c + 1]);
        // A zero scale's log2 is -inf: weight 0. So has a row that does not see the
        // key, whose scale may then be anything.
        w[c / 2] = pack_f16x2(t[c] == -INFINITY ? 0.0f : ex2_approx_ftz(t[c] + (st.rl[col + c] + lv)),
                              t[c + 1] == -INFINITY ? 0.0f : ex2_approx_ftz(t[c + 1] + (st.rl[col + c + 1] + lv)));
      }
    }
    if (!o_free && tc > 0) mbar_wait(at.p_empty, (tc - 1) & 1, dead);  // P^T's old contents are used
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(p_line + (((half * 4 + k) ^ (mine & 7)) << 4)) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    fence_async();
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(at.p_full);
  }
  if (n > 0) mbar_wait(at.p_empty, (tiles_done + n - 1) & 1, dead);
  tc_after();
  float* lsum = reinterpret_cast<float*>(at.ring_ptr);  // every operand has been used
#pragma unroll
  for (int c = 0; c < 32; c += 4)
    *reinterpret_cast<float4*>(lsum + mine * R + col + c) = make_float4(l[c], l[c + 1], l[c + 2], l[c + 3]);
}

// The item's result, by the softmax warps: the rows' sums, then O^T from TMEM.
template <int D, bool SHARED, bool HALF>
__device__ __noinline__ void wide_result() {
  using C = Wide<D, SHARED>;
  constexpr int R = C::R;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  const WideItem& item = st.item;
  volatile int32_t* dead = &st.dead;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c0 = item.c0;
  const int n = item.n;
  const int quarter = warp & 3, half = warp >> 2, mine = quarter * 32 + lane;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const int col = half * 32;
  const float* lsum = reinterpret_cast<const float*>(places<C>().ring_ptr);
  // NaN that the producers took out of rows that only some queries see: the
  // first such row (for shared rows: of any column) decides who gets it.
  const int64_t mixed0 = max(c0 * 128, (int64_t)(item.least / 128) * 128);
  const int64_t mixed1 = min((c0 + n) * 128, (int64_t)item.most);
  const bool nans = st.nan_rows != 0;
  if (nans && SHARED)
    for (int64_t key = mixed0 + threadIdx.x; key < mixed1; key += C::SW * 32) {
      const int32_t page = __ldg(item.row_table + (key >> item.page_bits));
      if (page < 0 || page >= item.num_pages) continue;
      const uint8_t* p = item.data +
                         ((((int64_t)page * item.heads + item.key_head) << item.page_bits) + (key & ((1 << item.page_bits) - 1))) * D;
      uint32_t any = 0;
      for (int k = 0; k < D; k += 4) any |= nan_bytes(__ldg(reinterpret_cast<const uint32_t*>(p + k)));
      if (any) atomicMin(&st.first_nan, (int)key);
    }
  barrier_of(3, C::SW * 32);
  constexpr int PARTS = C::SW * 32 / R;  // threads of a row's sum
  float part = 0.0f;
#pragma unroll 8
  for (int k = 0; k < 128 / PARTS; ++k)
    part += lsum[((threadIdx.x / R) * (128 / PARTS) + k) * R + threadIdx.x % R];
  st.part[threadIdx.x] = part;
  barrier_of(3, C::SW * 32);
  if (threadIdx.x < R) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) x += st.part[k * R + threadIdx.x];
    if ((SHARED && st.sees[threadIdx.x] > st.first_nan && st.row_at[threadIdx.x] >= 0) || *dead) x = NAN;
    RowStats r = {st.mref[threadIdx.x], st.mpref[threadIdx.x], x};
    st.factor[threadIdx.x] = out_factor(r);
    if (item.whole) {
      if (item.lse && st.row_at[threadIdx.x] >= 0) item.lse[st.row_at[threadIdx.x]] = row_lse(r);
    } else {
      *reinterpret_cast<float4*>(item.ws + R * D + threadIdx.x * 4) = make_float4(r.m, r.mp, r.l, 0.0f);
    }
  }
  barrier_of(3, C::SW * 32);
  for (int pp = 0; pp < C::PP; ++pp) {
    const int d = pp * 128 + mine;
    if (pp * 128 + quarter * 32 >= D) continue;  // the second copy of 64 columns
    int bad = 0x7FFFFFFF;  // first row whose value in column d is NaN
    if (nans && !SHARED)
      for (int64_t key = mixed0; key < mixed1; ++key) {
        const int32_t page = __ldg(item.row_table + (key >> item.page_bits));
        if (page < 0 || page >= item.num_pages) continue;
        const uint8_t byte = __ldg(
            item.data +
            ((((int64_t)page * item.heads + item.value_head) << item.page_bits) + (key & ((1 << item.page_bits) - 1))) * D + d);
        if ((byte & 0x7F) == 0x7F) {
          bad = (int)key;
          break;
        }
      }
    {
      float v[32];
      if (n > 0) {
        tc_load32(st.tmem + lanes + C::O0 + pp * R + col, v);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = 0.0f;
      }
      if (bad != 0x7FFFFFFF) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (st.sees[col + c] > bad) v[c] = NAN;
      }
      if (item.whole) {
        // neighbouring lanes trade rows, so that each stores two columns
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float fa = st.factor[col + c], fb = st.factor[col + c + 1];
          const float x = fa == 0.0f ? 0.0f : v[c] * fa, y = fb == 0.0f ? 0.0f : v[c + 1] * fb;
          const float other = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? x : y, 1);
          const uint32_t o = lane & 1 ? (HALF ? pack_f16x2(other, y) : pack_bf16x2(other, y))
                                      : (HALF ? pack_f16x2(x, other) : pack_bf16x2(x, other));
          const int64_t at = st.row_at[col + c + (lane & 1)];
          if (at >= 0) *reinterpret_cast<uint32_t*>(item.out + at * D + (d & ~1)) = o;
        }
      } else {  // slot 0: the item began with another worker, slot 1: it did here
        float* ws = item.ws + d;
#pragma unroll
        for (int c = 0; c < 32; ++c) ws[(col + c) * D] = v[c];
      }
    }
  }
  tc_before();
}

// What a producer's thread has stored of a panel: zeros where its mask says that
// the key is not there, and (`nans`) zeros for NaN, which it takes note of.
template <int D, bool SHARED>
__device__ __noinline__ void wide_clean(uint8_t* panel, int chunk, int kb, int pw, uint32_t here, bool nans) {
  using C = Wide<D, SHARED>;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
#pragma unroll 1
  for (int k = 0; k < C::KV; ++k) {
    const int e = C::step_of(k, pw), c16 = ((chunk & 3) * 2) ^ ((e * 4 + kb) & 7);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      uint4* v = reinterpret_cast<uint4*>(panel + e * 512 + ((c16 ^ i) << 4));
      uint4 x = *v;
      auto clean = [&](uint32_t w) -> uint32_t {  // fp16: an e4m3 NaN is all ones but the sign
        uint32_t keep = 0;
        if ((w & 0x7C00u) != 0x7C00u) keep |= 0xFFFFu;
        if ((w & 0x7C000000u) != 0x7C000000u) keep |= 0xFFFF0000u;
        if (keep != 0xFFFFFFFFu) st.nan_rows = 1;
        return w & keep;
      };
      if (!((here >> k) & 1))
        x = make_uint4(0, 0, 0, 0);
      else if (nans)
        x = make_uint4(clean(x.x), clean(x.y), clean(x.z), clean(x.w));
      *v = x;
    }
  }
}

// The producers. In a warp's load 4 keys x 8 chunks of 16 bytes; a store's
// quarter warp covers 2 keys x 4 chunks, which the swizzle spreads over all
// banks. Pages are looked up four planes at a time, a set ahead.
template <int D, bool SHARED>
__device__ __noinline__ void wide_produce() {
  using C = Wide<D, SHARED>;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  const Places<C> at = places<C>();
  const WideItem& item = st.item;
  volatile int32_t* dead = &st.dead;
  const int lane = threadIdx.x & 31, pw = (threadIdx.x >> 5) - C::SW;
  const int64_t c0 = item.c0;
  const int n = item.n, most = item.most, least = item.least;
  const Planes<SHARED> planes = {n};
  const int chunk = (lane & 3) | ((lane >> 1) & 4);
  const int kb = ((lane >> 2) & 1) | ((lane >> 3) & 2);  // this thread's of a step's 4 keys
  // 16 keys in a row lie on one page. Lane 8 p + g holds the page of keys 16 g ..
  // of plane 4 m + p.
  auto pages_of = [&](int m) -> int32_t {
    const int q = 4 * m + (lane >> 3);
    if (q >= planes.count()) return -1;
    const int64_t key = (c0 + planes.tile(q)) * 128 + (lane & 7) * 16;
    return key < most ? __ldg(item.row_table + (key >> item.page_bits)) : -1;
  };
  int32_t pages = pages_of(0), pages_next = pages_of(1);
  // Lanes 8 p + g: where the 16 keys begin, in KiB from the pool's start, or -1.
  auto locate16 = [&](int m, int32_t page) -> int32_t {
    const int q = 4 * m + (lane >> 3);
    if (page < 0 || page >= item.num_pages) return -1;
    const int64_t key = (c0 + planes.tile(q)) * 128 + (lane & 7) * 16;
    const int head = planes.value(q) ? item.value_head : item.key_head;
    const int slot = (int)(key & ((1 << item.page_bits) - 1));
    return (int32_t)((((((int64_t)page * item.heads + head) << item.page_bits) + slot) * D) >> 10);
  };
  int32_t kib = locate16(0, pages), kib_next = -1;
  int line[C::KV];  // where the step's first 8 values go in a panel
#pragma unroll
  for (int k = 0; k < C::KV; ++k) {
    const int e = C::step_of(k, pw);
    line[k] = (chunk >> 2) * C::SLAB + (e * 4 + kb) * 128 + ((((chunk & 3) * 2) ^ ((e * 4 + kb) & 7)) << 4);
  }
  const uint8_t* const pool = item.data;
  const uint8_t* src[C::KV];
  uint4 buf[C::DEPTH][C::KV];
  uint32_t here[C::DEPTH];  // bit k: the key of step k is there; the others are loaded from
                            // the pool's start and stored as zeros
  int load_q = 0, load_pp = 0;
  uint32_t there = 0;
  auto load = [&](uint4 (&v)[C::KV], uint32_t& mask) {  // the next panel of the sequence
    if (load_pp == 0) {
      const int m = load_q >> 2, p = load_q & 3;
      if (p == 0 && load_q > 0) {
        kib = kib_next;
      } else if (p == 1) {  // the lookup of the next four has had four planes' time
        kib_next = locate16(m + 1, pages_next);
        pages_next = pages_of(m + 2);
      }
      const int left = load_q < planes.count()
                           ? (int)min((int64_t)128, (int64_t)most - (c0 + planes.tile(load_q)) * 128)
                           : 0;
      there = 0;
#pragma unroll
      for (int k = 0; k < C::KV; ++k) {
        const int e = C::step_of(k, pw);
        const int32_t first = __shfl_sync(0xFFFFFFFFu, kib, p * 8 + (e >> 2));
        const bool ok = first >= 0 && e * 4 + kb < left;
        there |= (uint32_t)ok << k;
        src[k] = pool + (ok ? (int64_t)first << 10 : 0) + ((e & 3) * 4 + kb) * D + (chunk * 16) % D;
      }
    }
    mask = there;
#pragma unroll
    for (int k = 0; k < C::KV; ++k)
      v[k] = ld_stream(reinterpret_cast<const uint16_t*>(src[k] + load_pp * 128));
    if (++load_pp == C::PP) {
      load_pp = 0;
      ++load_q;
    }
  };
#pragma unroll
  for (int j = 0; j < C::DEPTH; ++j) load(buf[j], here[j]);
  const int total = planes.count() * C::PP;
  const uint32_t panels_done = item.panels_done;
  uint8_t* const ring = at.ring_ptr;
  for (int p0 = 0; p0 < total; p0 += C::DEPTH) {
#pragma unroll
    for (int j = 0; j < C::DEPTH; ++j) {
      const int p = p0 + j;
      if (p >= total) break;
      const uint32_t pc = panels_done + p, slot = pc % C::NS;
      const int q = p / C::PP;
      // Heads of several panels: widened before the slot is free, since the refill of
      // the ring is what the matrix instructions wait for (latent rows 191 -> 189 us).
      // With one panel ahead the data would be waited for too early (80 -> 82.5 us).
      const uint32_t freed = at.empty + 8 * slot, phase = ((pc / C::NS) & 1) ^ 1;
      if (C::PP == 1) mbar_wait(freed, phase, dead);
      uint4 wide[C::KV][2];
#pragma unroll
      for (int k = 0; k < C::KV; ++k) {
        const uint4 x = buf[j][k];
        wide[k][0] = make_uint4(lo_f16x2(x.x), hi_f16x2(x.x), lo_f16x2(x.y), hi_f16x2(x.y));
        wide[k][1] = make_uint4(lo_f16x2(x.z), hi_f16x2(x.z), lo_f16x2(x.w), hi_f16x2(x.w));
      }
      const uint32_t there_now = here[j];
      if (C::PP > 1) mbar_wait(freed, phase, dead);
      uint8_t* panel = ring + slot * C::PANEL;
#pragma unroll
      for (int k = 0; k < C::KV; ++k) {
        *reinterpret_cast<uint4*>(panel + line[k]) = wide[k][0];
        *reinterpret_cast<uint4*>(panel + (line[k] ^ 16)) = wide[k][1];
      }
      // Missing rows become zeros, and rows that only some queries see must not
      // bring NaN into the product: both rare.
      const bool mixed = (SHARED || planes.value(q)) && (c0 + planes.tile(q) + 1) * 128 > least;
      if (mixed || there_now != (1u << C::KV) - 1)
        wide_clean<D, SHARED>(panel + (chunk >> 2) * C::SLAB + kb * 128, chunk, kb, pw, there_now, mixed);
      load(buf[j], here[j]);  // while the stores are under way
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(at.full + 8 * slot);
    }
  }
}

template <int D, bool SHARED, bool HALF>
__global__ void __launch_bounds__(Wide<D, SHARED>::THREADS, 1)
    attend_wide_kernel(const AttendArgs a, const PlanShape plan) {
  using C = Wide<D, SHARED>;
  auto& st = *reinterpret_cast<typename C::State*>(wide_smem);
  grid_dependency_wait();
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5;
  const Place place = locate<C::THREADS>(a, plan, blockIdx.x, st.sums, &st.found);
  Shared* left = shared_items<C::R, D>(a, plan.workers) + blockIdx.x;  // unless items are whole
  if (place.pos < 0) {
    if (threadIdx.x == 0 && !plan.whole) left->parts = 0;
    return;
  }
  Shared tail = {0, 0, 0, 0};  // an item that begins here and ends with another worker
  const Places<C> at = places<C>();
  if (threadIdx.x == 0) {
    st.dead = 0;
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(at.full + 8 * i, C::PW);
      mbar_init(at.empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(at.s_full + 8 * i, 1);
      mbar_init(at.s_empty + 8 * i, C::SW);
    }
    mbar_init(at.p_full, C::SW);
    mbar_init(at.p_empty, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::SW) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_at(&st.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();

  uint32_t panels_done = 0, tiles_done = 0;
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
    const int64_t tile_of_rows = item - h * work.tiles;
    const int64_t units = plan.whole ? 1 : min(work.chunks - c0, place.end - pos);
    const int64_t c1 = plan.whole ? (int64_t)1 << 40 : c0 + units;
    const bool whole = plan.whole || units == work.chunks;
    if (c0 == 0 && !whole)
      tail = {1 + (int32_t)((work.chunks - c1 + place.per - 1) / place.per), s, (int32_t)tile_of_rows, h};

    // ---- the rows: what they see, and Q as fp16 --------------------------------
    if (threadIdx.x == 0) {
      st.sees_least = 0x7FFFFFFF;
      st.sees_most = 0;
      for (int k = 0; k < C::R / 32; ++k) st.far_refs[k] = 0;
      st.nan_rows = 0;
      st.first_nan = 0x7FFFFFFF;
    }
    __syncthreads();
    stage_rows<D, SHARED>(a, s, tile_of_rows, h, work.keys);
    __syncthreads();
    const int64_t stop = min(c1, ((int64_t)st.sees_most + 127) / 128);
    const int n = stop > c0 ? (int)(stop - c0) : 0;  // tiles of 128 keys
    if (threadIdx.x == 0) {
      WideItem& it = st.item;
      it.data = a.c.data;
      it.scales = a.c.scales;
      it.row_table = a.table + (int64_t)s * a.max_pages;
      it.ws = a.ws + ((int64_t)blockIdx.x * 2 + (c0 == 0)) * C::SLOT;
      it.out = a.out;
      it.lse = a.lse;
      it.c0 = c0;
      it.n = n;
      it.least = st.sees_least;
      it.most = st.sees_most;
      it.key_head = h;
      it.value_head = a.v_first + h;
      it.heads = a.c.heads;
      it.num_pages = a.c.num_pages;
      it.page_bits = a.c.page_bits;
      it.block_bits = a.c.block_bits;
      it.panels_done = panels_done;
      it.tiles_done = tiles_done;
      it.whole = whole;
    }
    __syncthreads();
    if (warp < C::SW) {
      stage_queries<D, SHARED, HALF>(a.q, a.scale);
      fence_async();
      barrier_of(4, C::SW * 32 + 32);  // Q is there, for the warp of the matrix instructions
      wide_softmax<D, SHARED>();
      wide_result<D, SHARED, HALF>();
    } else if (warp < C::SW + C::PW) {
      wide_produce<D, SHARED>();
    } else {
      barrier_of(4, C::SW * 32 + 32);
      wide_products<D, SHARED>();
    }
    __syncthreads();
    panels_done += (SHARED ? 1 : 2) * n * C::PP;
    tiles_done += n;
    pos += units;
    within += units;
  }
  if (threadIdx.x == 0 && !plan.whole) *left = tail;
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == C::SW)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(st.tmem) : "memory");
}

template <int D, bool SHARED, bool HALF>
cudaError_t launch_wide(AttendArgs a, cudaStream_t stream) {
  using C = Wide<D, SHARED>;
  static_assert(C::each_step_by_one_warp(), "producer warps share keys of a panel");
  const PlanShape p = plan_of(a, C::R, 128, 152, 2, 8, 0);
  auto* kernel = attend_wide_kernel<D, SHARED, HALF>;
  cudaError_t e = allow_dynamic_smem((const void*)kernel, C::SMEM);
  if (e != cudaSuccess) return e;
  if (p.whole)
    return launch_dependent(kernel, dim3((unsigned)p.workers), dim3(C::THREADS), C::SMEM, stream, a, p);
  void* ws = nullptr;
  e = workspace_take(&ws, join_bytes<D, C::R>(p.workers), stream);
  if (e != cudaSuccess) return e;
  a.ws = static_cast<float*>(ws);
  e = launch_dependent(kernel, dim3((unsigned)p.workers), dim3(C::THREADS), C::SMEM, stream, a, p);
  if (e == cudaSuccess) e = launch_join<D, C::R, HALF>(a, p.workers, stream);
  const cudaError_t ef = workspace_give(ws, stream);
  return e != cudaSuccess ? e : ef;
}

template <int D>
cudaError_t launch_dim(const AttendArgs& a, bool half, bool shared, cudaStream_t stream) {
  if (shared) return half ? launch_wide<D, true, true>(a, stream) : launch_wide<D, true, false>(a, stream);
  return half ? launch_wide<D, false, true>(a, stream) : launch_wide<D, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_attend_wide(const AttendArgs& a, bool half, bool shared, cudaStream_t stream) {
  switch (a.c.d) {
    case 64: return launch_dim<64>(a, half, shared, stream);
    case 128: return launch_dim<128>(a, half, shared, stream);
    case 256: return launch_dim<256>(a, half, shared, stream);
    default: return launch_dim<512>(a, half, shared, stream);
  }
}

}  // namespace csa
