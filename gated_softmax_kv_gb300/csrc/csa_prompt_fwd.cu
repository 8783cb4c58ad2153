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
// instructions, one for TMA, one that finds the work. Tiles of K and V come in a ring,
// in the order in which the instructions use them. Where only one tile has rows (single
// tokens, short prompts) both softmax groups work on it, on alternate blocks of keys,
// and add up at the end.
//
// A CTA that is done takes over the work of one that has not started (cluster launch
// control), so that the copies and first products of its next item run beside the
// result of this one. Grids that leave SMs idle are launched as clusters instead,
// whose CTAs share an item's keys and add up through distributed shared memory.
//
// The reference that logits are taken from rises only when they pass it by 2^8, so
// that O is seldom scaled: weights are at most 2^8. fp16 weights are lifted by
// another 2^7, so that small ones keep their bits; the factor cancels. Sums of
// weights are of what is not rounded yet.
//
// Blocks that some row of the CTA does not see in full are cleaned of infinities and
// NaN in V, which a weight of 0 would not keep out, by a warp of its own; rows that do
// see one get it back from memory at the end.
//
// What bounds it: on long keys the tensor core under the power limit, 16384 tokens of 16
// heads over 2 of 128 columns 642 to 737 us by the box (1710 to 1490 TFLOP/s; 2048 cycles of
// products in 2400 of a round of both tiles). An item costs about 4 us beside its blocks: 12
// ragged sequences of up to 2047 tokens, 32 heads over 8, 159 us (954 TFLOP/s); a window of
// 128 over 5003 tokens of 64 heads of 64, 92 us. Single tokens: memory, 32 sequences of 8192
// keys, 8 key heads of 128, 158 us (6.8 TB/s).
//
// Every wait on an mbarrier is bounded (csa_prompt_tile.cuh): a wait that runs out marks the
// CTA, whose later waits return at once and whose unfinished items' results become NaN.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "csa_internal.h"
#include "csa_prompt_tile.cuh"

namespace csa {

namespace {

template <int DP_, bool HALF_, bool WINDOW_>
struct Fwd {
  static constexpr int DP = DP_;                  // columns, padded to a slab of 64
  static constexpr bool HALF = HALF_;
  static constexpr bool WINDOW = WINDOW_;
  static constexpr int SLAB = 16384;              // 128 rows x 64 columns
  static constexpr int TILE = DP / 64 * SLAB;
  static constexpr int NS = DP == 128 ? 5 : 8;    // tiles of the ring
  static constexpr int SHARE = DP + 4;            // floats of a row that a cluster shares
  static_assert(128 * SHARE * 4 <= NS * TILE, "a cluster shares its sums in the ring");
  static constexpr int THREADS = 384;
  // Registers: 384 threads at 168, dealt out again by role (2 * 208 + 88 = 3 * 168).
  static constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;
  static constexpr int HEAD = 2048;  // barriers and the item
  static constexpr int SMEM = 1024 + HEAD + (2 + NS) * TILE;
  static constexpr uint32_t S0 = 0, O0 = 256;     // TMEM columns: S of the two tiles, O of the two
  static constexpr uint32_t TYPES = HALF ? 0u : (1u << 7) | (1u << 10);
  // fp32 accumulator, M = 128; N = 128 keys; N = DP columns, the second operand N-major
  static constexpr uint32_t IDESC_S = (1u << 4) | TYPES | ((128u >> 3) << 17) | (8u << 24);
  static constexpr uint32_t IDESC_O = (1u << 4) | TYPES | (1u << 16) | ((uint32_t)(DP >> 3) << 17) | (8u << 24);
  static constexpr float LIFT = HALF ? 7.0f : 0.0f;
};

// An item of work: the query rows of up to two tiles, and the keys that they see.
struct alignas(16) Item {
  int32_t q0, nq, k0, off;   // first row of the sequence in q and k; its queries; key index of query 0
  int32_t t0, last;          // first and last token
  int32_t kvh;               // key head
  int32_t kb0, n0, n1, step; // first block of keys, blocks of each tile, 2: the groups share tile 0
  int32_t pad;               // n0 < 0: there is no more work
  __device__ __forceinline__ bool keys() const { return n0 > 0 || n1 > 0; }
};

template <int NS>
struct State {
  Item item[2];
  WorkState work;
  uint64_t full[NS], empty[NS], q_full, q_empty, s_full[2], p_full[2][2], o_full[2], pair_full, pair_empty, clean[NS];
  int32_t dead, bad;
  uint32_t tmem;
  float ref[128], sum[128];  // group 1's, for group 0; in a cluster: the CTA's
};

// The order of the ring: K0 V0 K1 V1 ... or, where the groups take alternate blocks, K0
// K1 V0 K2 V1 ...: the block of an item's i-th tile, and whether it is of values.
__device__ __forceinline__ int tile_at(int i, int n, int step, bool& value) {
  if (step == 1) {
    value = i & 1;
    return i / 2;
  }
  value = i == 2 * n - 1 || (i > 1 && (i & 1) == 0);
  return i == 2 * n - 1 ? n - 1 : value ? i / 2 - 1 : (i + 1) / 2;
}

// The blocks [from, to) that every row of tokens ta .. tb sees in full.
struct Seen {
  int from, to;
  __device__ __forceinline__ bool all(int b) const { return b >= from && b < to; }
};
__device__ __forceinline__ Seen seen_by(const PromptArgs& a, const Item& x, int ta, int tb) {
  Seen s;
  s.to = max(x.off + ta + 1, 0) / 128 - x.kb0;
  s.from = a.window ? (int)((max((int64_t)x.off + tb + 1 - a.window, (int64_t)0) + 127) / 128) - x.kb0 : 0;
  return s;
}

extern __shared__ __align__(1024) uint8_t fwd_smem[];

// Infinities and NaN of V that were cleaned away, for 32 columns of a row that sees
// keys lo .. hi - 1.
template <bool HALF>
__device__ __noinline__ void give_back(const PromptArgs& a, const Item& x, int lo, int hi, int col, float* o) {
  const Seen seen = seen_by(a, x, x.t0, x.last);
#pragma unroll 1
  for (int b = 0; b < max(x.n0, x.n1); ++b) {
    if (seen.all(b)) continue;
    const int k0 = max(lo, (x.kb0 + b) * 128), k1 = min(hi, (x.kb0 + b) * 128 + 128);
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      const uint16_t* v = static_cast<const uint16_t*>(a.v) + (int64_t)(x.k0 + k) * a.vt + x.kvh * a.vh + col;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (col + c < a.d) {
          const float f = value16<HALF>(__ldg(v + c));
          if (!isfinite(f)) o[c] += f;
        }
    }
  }
}

// How a launch deals out its work.
struct FwdShape {
  int32_t tiles;  // of a CTA: 1 or 2
  int32_t split;  // CTAs that share an item's keys: a cluster
};

// Item `id`, by a warp; n0 < 0 where the slot has none. Later slots first: a sequence's
// last tiles see the most keys.
__device__ __forceinline__ Item item_of(const PromptArgs& a, const FwdShape& shape, uint32_t id, uint32_t ids, int part,
                                        int lane) {
  Item x;
  const int tp = 128 / a.group, b = shape.tiles * tp;
  id = ids - 1 - id;
  const int64_t slot = id / a.kv;
  x.kvh = (int)(id - slot * a.kv);
  const int s = seq_of_slot(a.cu_q, a.nseq, b, slot, lane);
  const Span w = span_of<false>(a, s);
  const int64_t local = slot - first_slot(a.cu_q, s, b);
  x.q0 = w.q0;
  x.nq = w.nq;
  x.k0 = w.k0;
  x.off = w.nk - w.nq;
  x.n0 = -1;
  x.n1 = 0;
  if (local < 0 || local * b >= w.nq) return x;
  x.t0 = (int)local * b;
  x.last = min(x.t0 + b, w.nq) - 1;
  x.kb0 = (a.window ? (int)max((int64_t)0, (int64_t)x.off + x.t0 + 1 - a.window) : 0) / 128;
  auto blocks = [&](int ta) {
    const int tb = min(ta + tp - 1, x.last), end = x.off + tb + 1;
    return tb >= ta && end > 0 ? (end + 127) / 128 - x.kb0 : 0;
  };
  x.n0 = blocks(x.t0);
  x.n1 = blocks(x.t0 + tp);
  x.step = 1;
  if (shape.split > 1) {
    const int per = (x.n0 + shape.split - 1) / shape.split;
    x.kb0 += part * per;
    x.n0 = max(0, min(per, x.n0 - part * per));
  }
  if (x.t0 + tp > x.last && x.n0 > 1) {
    x.step = 2;
    x.n1 = x.n0;
  }
  return x;
}

// 32 columns of a row of a result.
template <class C>
__device__ __forceinline__ void put_columns(const PromptArgs& a, int64_t row, int k, const float* o) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack16<C::HALF>(o[2 * i], o[2 * i + 1]);
  auto put = [&](void* to) {
    uint16_t* p = static_cast<uint16_t*>(to) + row * a.d + k;
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0 && a.d % 16 == 0) {  // tensors are 16-byte aligned at least
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (k + 16 * i < a.d) st_sector(p + 16 * i, w + 8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k + 8 * i < a.d)
          *reinterpret_cast<uint4*>(p + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  };
  put(a.out);
  if (a.rest) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i] = pack16<C::HALF>(o[2 * i] - value16<C::HALF>((uint16_t)w[i]), o[2 * i + 1] - value16<C::HALF>((uint16_t)(w[i] >> 16)));
    put(a.rest);
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prompt_fwd_kernel(const __grid_constant__ PromptArgs a, const FwdShape shape, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* const base = fwd_smem + ((1024u - (smem_at(fwd_smem) & 1023u)) & 1023u);
  auto& st = *reinterpret_cast<State<C::NS>*>(base);
  static_assert(sizeof(State<C::NS>) <= C::HEAD, "HEAD");
  uint8_t* const q_ptr = base + C::HEAD;
  uint8_t* const ring_ptr = q_ptr + 2 * C::TILE;
  const uint32_t q_at = smem_at(q_ptr), ring = smem_at(ring_ptr);
  const uint32_t full = smem_at(st.full), empty = smem_at(st.empty), q_full = smem_at(&st.q_full),
                 q_empty = smem_at(&st.q_empty), s_full = smem_at(st.s_full), p_full = smem_at(st.p_full),
                 o_full = smem_at(st.o_full), pair_full = smem_at(&st.pair_full), pair_empty = smem_at(&st.pair_empty),
                 clean = smem_at(st.clean);
  const Dead dead = {&st.dead, a.polls};
  const int tp = 128 / a.group, rows = tp * a.group;
  const uint32_t ids = gridDim.x / shape.split, first_id = blockIdx.x / shape.split;
  const int part = (int)(blockIdx.x - first_id * shape.split);  // of the item, in a cluster
  if (threadIdx.x == 0) {
    st.dead = st.bad = 0;
#pragma unroll 1
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 2);  // the matrix instructions and the cleaning warp
      mbar_init(clean + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(pair_full, 4);
    mbar_init(pair_empty, 4);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + 8 * t, 1);
      mbar_init(p_full + 16 * t, 4);
      mbar_init(p_full + 16 * t + 8, 4);
      mbar_init(o_full + 8 * t, 1);
    }
    init_work(st.work, 11);  // eight softmax warps, copies, cleaning, matrix instructions
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
    if (warp == 10) {  // ---- work
      find_work(st.work, st.item, first_id, shape.split > 1, lane, dead, [&](uint32_t id) {
        if (part == 0) {  // this item's share of the rows of no sequence
          const int64_t from = (int64_t)id * 32 + lane, step = (int64_t)ids * 32;
          if (a.fill & CSA_FILL_OUT) {
            const int64_t words = (int64_t)a.heads * a.d / 8;
            fill_rest(a.cu_q, a.nseq, a.num_q, words, static_cast<uint4*>(a.out), from, step);
            if (a.rest) fill_rest(a.cu_q, a.nseq, a.num_q, words, static_cast<uint4*>(a.rest), from, step);
          }
          if (a.fill & CSA_FILL_LSE) fill_rest(a.cu_q, a.nseq, a.num_q, a.heads, -INFINITY, a.lse, from, step);
        }
        return item_of(a, shape, id, ids, part, lane);
      });
    } else if (warp == 11) {  // ---- infinities and NaN of values that not every row sees
      // Every tile of the ring is waited for, keys too, and its place is held until this warp
      // has seen it: a parity tells only whether the tile before it in its place has come.
      Place<C::NS> at = {0, 0};
#pragma unroll 1
      for (int k = 0;; ++k) {
        const Item x = take(k);
        if (x.n0 < 0) break;
        const int n = max(x.n0, x.n1);
        const Seen seen = seen_by(a, x, x.t0, x.last);
#pragma unroll 1
        for (int i = 0; i < 2 * n; ++i) {
          bool value;
          const int b = tile_at(i, n, x.step, value);
          wait_for(full + 8 * at.stage, at.parity, dead);
          if (value && !seen.all(b)) {
            clean_operand<C::HALF>(ring_ptr + at.stage * C::TILE, C::TILE, lane, &st.bad);
            __syncwarp();
            if (lane == 0) mbar_arrive(clean + 8 * at.stage);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty + 8 * at.stage);
          tile_seen(st.work, lane);
          at.next(1);
        }
      }
    } else if (warp == 9) {  // ---- copies
      Place<C::NS> at = {0, 0};
      uint32_t loaded = 0;  // items with keys
      uint32_t copies = 0;
      if (lane == 0) {
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
      }
#pragma unroll 1
      for (int k = 0;; ++k) {
        const Item x = take(k);
        if (x.n0 < 0) break;
        const int n = max(x.n0, x.n1);
        if (n == 0) continue;
        if (lane == 0) wait_for(q_empty, (loaded & 1) ^ 1, dead);
        if (lane == 0 && !*dead) {
          const int tiles = x.step == 1 && x.n1 > 0 ? 2 : 1;
          mbar_expect(q_full, tiles * (C::DP / 64) * 128 * rows);
#pragma unroll 1
          for (int t = 0; t < tiles; ++t)
#pragma unroll 1
            for (int p = 0; p < C::DP / 64; ++p)
              tma_load(q_at + t * C::TILE + p * C::SLAB, &mq, p * 64, x.kvh * a.group, x.q0 + x.t0 + t * tp, q_full);
#pragma unroll 1
          for (int i = 0; i < 2 * n; ++i) {
            bool value;
            const int b = tile_at(i, n, x.step, value);
            wait_for(empty + 8 * at.stage, at.parity ^ 1, dead);
            if (*dead) break;
            mbar_expect(full + 8 * at.stage, C::TILE);
#pragma unroll 1
            for (int p = 0; p < C::DP / 64; ++p)
              tma_load(ring + at.stage * C::TILE + p * C::SLAB, value ? &mv : &mk, p * 64, x.kvh, x.k0 + (x.kb0 + b) * 128,
                       full + 8 * at.stage);
            ++copies;
            at.next(1);
          }
          ++loaded;
        }
        __syncwarp();
      }
      if (lane == 0) {
        land_ring(full, C::NS, copies);
        land_ring(q_full, 1, loaded);
      }
    } else if (warp == 8) {  // ---- matrix instructions
      // Issuing them is a warp's whole work: what it counts stays in registers, with no
      // divisions and no waits that are known to have passed (a tile 1900 -> 1100 cycles).
      const uint32_t leader = tc_leader(), tm = uniform(tmem);
      const uint64_t q_op = operand(q_at, 16), k_op = operand(ring, 16), v_op = operand(ring, C::SLAB);
      Place<C::NS> start = {0, 0};
      uint32_t loaded = 0, copies = 0, cleaned = 0, rounds[2] = {0, 0};  // cleaned: a parity a stage
#pragma unroll 1
      for (int k = 0;; ++k) {
        const Item x = take(k);
        const int n0 = (int)uniform((uint32_t)x.n0), n1 = (int)uniform((uint32_t)x.n1), step = (int)uniform((uint32_t)x.step);
        if (n0 < 0) break;
        const int n = max(n0, n1);
        if (n == 0) continue;
        const Seen seen = seen_by(a, x, x.t0, x.last);
        const int seen_from = (int)uniform((uint32_t)seen.from), seen_to = (int)uniform((uint32_t)seen.to);
        wait_for(q_full, loaded & 1, dead);
        ++loaded;
        // keys and values of the next block to come, of either tile
        Place<C::NS> key = start, value = start;
        value.next(step);
        auto scores = [&](int t, int at) {  // S of tile t and the keys at a place of the ring
          const uint64_t q = q_op + (step == 1 ? t : 0) * (C::TILE / 16), kk = k_op + at * (C::TILE / 16);
#pragma unroll
          for (int p = 0; p < C::DP / 64; ++p)
            tc_mma4<2>(leader, tm + C::S0 + 128 * t, q + p * (C::SLAB / 16), kk + p * (C::SLAB / 16), C::IDESC_S, p > 0);
          tc_commit_by(leader, s_full + 8 * t);
        };
        auto ready = [&](const Place<C::NS>& p) {
          wait_for(full + 8 * p.stage, p.parity, dead);
          tc_after();
        };
        auto valued = [&](int b) {  // the values of block b are there, and clean
          ready(value);
          if (b < seen_from || b >= seen_to) {
            wait_for(clean + 8 * value.stage, (cleaned >> value.stage) & 1, dead);
            cleaned ^= 1u << value.stage;
            tc_after();
          }
        };
        auto weigh = [&](int t, int at, bool first) {  // O of tile t += its weights and the values at a place
          const uint64_t v = v_op + at * (C::TILE / 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wait_for(p_full + 16 * t + 8 * h, rounds[t] & 1, dead);
            tc_after();
            tc_mma4_ts<128>(leader, tm + C::O0 + C::DP * t, tm + C::S0 + 128 * t + 32 * h, v + 512 * h, C::IDESC_O, !first || h > 0);
          }
          ++rounds[t];
        };
        ready(key);
        if (step == 1) {
          if (n0 > 0) scores(0, key.stage);
          if (n1 > 0) scores(1, key.stage);
          tc_commit_by(leader, empty + 8 * key.stage);
          if (n == 1) tc_commit_by(leader, q_empty);
          key.next(2);
#pragma unroll 1
          for (int b = 0; b < n; ++b) {
            if (b == max(0, n - 3)) want_work(st.work, lane);
            valued(b);
            const bool more = b + 1 < n;
            if (b < n0) {
              weigh(0, value.stage, b == 0);
              if (b + 1 < n0) {
                ready(key);
                scores(0, key.stage);
              } else {
                tc_commit_by(leader, o_full);
              }
            }
            if (b < n1) {
              weigh(1, value.stage, b == 0);
              tc_commit_by(leader, empty + 8 * value.stage);
              if (b + 1 < n1) {
                if (b + 1 >= n0) ready(key);
                scores(1, key.stage);
              } else {
                tc_commit_by(leader, o_full + 8);
              }
            } else {
              tc_commit_by(leader, empty + 8 * value.stage);
            }
            if (more) tc_commit_by(leader, empty + 8 * key.stage);
            if (b + 2 == n) tc_commit_by(leader, q_empty);
            key.next(2);
            value.next(2);
          }
        } else {  // n >= 2: tile 0 has the even blocks, 1 the odd ones
          scores(0, key.stage);
          tc_commit_by(leader, empty + 8 * key.stage);
          key.next(1);
          ready(key);
          scores(1, key.stage);
          tc_commit_by(leader, empty + 8 * key.stage);
          if (n == 2) tc_commit_by(leader, q_empty);
          key.next(2);
#pragma unroll 1
          for (int b = 0; b < n; b += 2) {
            if (b == (max(0, n - 6) & ~1)) want_work(st.work, lane);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (b + t >= n) break;
              valued(b + t);
              weigh(t, value.stage, b == 0);
              tc_commit_by(leader, empty + 8 * value.stage);
              value.next(b + t + 2 == n ? 1 : 2);
              if (b + t + 2 < n) {
                ready(key);
                scores(t, key.stage);
                tc_commit_by(leader, empty + 8 * key.stage);
                if (b + t + 3 == n) tc_commit_by(leader, q_empty);
                key.next(2);
              } else {
                tc_commit_by(leader, o_full + 8 * t);
              }
            }
          }
        }
        copies += 2 * n;
        start = {(int)(copies % C::NS), (copies / C::NS) & 1};
      }
      end_products(st.work, leader);
    }
  } else {  // ---- softmax and result: a row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + C::S0 + 128 * t, o_at = tmem + lanes + C::O0 + C::DP * t;
    const float c = a.scale * kLog2e;
    const int in_tile = r / a.group, head = r - in_tile * a.group;
    uint32_t rounds = 0, results = 0, pairs = 0;
#pragma unroll 1
    for (int k = 0;; ++k) {
      const Item x = take(k);
      if (x.n0 < 0) break;
      const int mine = t ? x.n1 : x.n0;
      const int ta = x.t0 + (x.step == 1 ? t * tp : 0), tb = min(ta + tp - 1, x.last);
      const int token = ta + in_tile;
      const bool there = r < rows && token <= tb;
      const int hi = there ? x.off + token + 1 : 0;
      const int lo = a.window ? (int)max((int64_t)0, (int64_t)x.off + token + 1 - a.window) : 0;
      const Seen seen = seen_by(a, x, ta, tb);
      float ref = -INFINITY;  // in log2 units
      float2 l0 = make_float2(0.0f, 0.0f), l1 = l0;
#pragma unroll 1
      for (int b = x.step == 1 ? 0 : t; b < mine; b += x.step) {
        wait_for(s_full + 8 * t, rounds & 1, dead);
        ++rounds;
        tc_after();
        float v[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tc_load32_async(s_at + 32 * i, v + 32 * i);
        tc_load_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) tc_loaded(v + 32 * i);
        // With a window, most of a block is hidden: which 32 columns some row of the warp
        // sees, the others cost nothing (5003 tokens of 64 heads of 64, window 128: 140 us, so
        // 95). Without one the branches cost more than they save (16384 tokens: 632 us, 674).
        uint32_t some_see = 15;
        if (!seen.all(b)) {
          const int k0 = (x.kb0 + b) * 128, h = hi - k0, w = lo - k0;
          if constexpr (C::WINDOW) some_see = 0;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if constexpr (C::WINDOW) {
              if (!__any_sync(0xFFFFFFFFu, h > 32 * g && w < 32 * g + 32 && h > w)) continue;
              some_see |= 1u << g;
            }
            if (!__any_sync(0xFFFFFFFFu, h < 32 * g + 32 || w > 32 * g)) continue;
            // bit i: column 32 g + i is seen
            const int from = max(w - 32 * g, 0), to = min(h - 32 * g, 32);
            const uint32_t bits = to > from ? (0xFFFFFFFFu >> (32 - (to - from))) << from : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[32 * g + i] = bits >> i & 1 ? v[32 * g + i] : -INFINITY;
          }
        }
        float m0 = -INFINITY, m1 = -INFINITY;
        auto largest = [&](int g) {
#pragma unroll
          for (int i = 32 * g; i < 32 * g + 32; i += 4) {
            m0 = fmaxf(m0, fmaxf(v[i], v[i + 1]));
            m1 = fmaxf(m1, fmaxf(v[i + 2], v[i + 3]));
          }
        };
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (!C::WINDOW || (some_see >> g & 1)) largest(g);
        const float z = fmaxf(m0, m1) * c;
        const bool raise = z > ref + 8.0f;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          const float f = raise ? ex2_approx_ftz(ref - z) : 1.0f;
          if (raise) ref = z;
          l0.x *= f;
          l0.y *= f;
          l1.x *= f;
          l1.y *= f;
          if (b >= x.step) {  // the products before are done: S of this block came after them
#pragma unroll 1
            for (int i = 0; i < C::DP; i += 32) {
              float o[32];
              tc_load32(o_at + i, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= f;
              tc_store32(o_at + i, o);
            }
          }
        }
        const float back = C::LIFT - (ref == -INFINITY ? 0.0f : ref);
        auto weights = [&](int g, bool any) {  // of 32 columns
          uint32_t p[16];
          if (any) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const int i = 32 * g + j;
              const float2 za = fma2_rn(make_float2(v[i], v[i + 1]), make_float2(c, c), make_float2(back, back));
              const float2 zb = fma2_rn(make_float2(v[i + 2], v[i + 3]), make_float2(c, c), make_float2(back, back));
              const float2 pa = make_float2(ex2_approx_ftz(za.x), ex2_approx_ftz(za.y));
              const float2 pb = make_float2(ex2_approx_ftz(zb.x), ex2_approx_ftz(zb.y));
              l0 = add2_rn(l0, pa);
              l1 = add2_rn(l1, pb);
              p[j / 2] = pack16<C::HALF>(pa.x, pa.y);
              p[j / 2 + 1] = pack16<C::HALF>(pb.x, pb.y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = 0;
          }
          tc_store16_async(s_at + 16 * g, p);
          if (g & 1) {  // 64 weights: their products begin
            tc_store_wait();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * (g / 2));
          }
        };
#pragma unroll
        for (int g = 0; g < 4; ++g) weights(g, !C::WINDOW || (some_see >> g & 1));
      }
      float l = (l0.x + l0.y) + (l1.x + l1.y);
      if (mine > 0) wait_for(o_full + 8 * t, results++ & 1, dead);
      tc_after();
      // O = fa O of tile 0 + fb O of tile 1, where both groups have worked on the same rows
      float fa = 1.0f, fb = 0.0f;
      if (x.step == 2) {
        if (t == 1) {
          st.ref[r] = ref;
          st.sum[r] = l;
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pair_full);
        } else {
          wait_for(pair_full, pairs & 1, dead);
          tc_after();
          const float other = st.ref[r], top = fmaxf(ref, other), safe = top == -INFINITY ? 0.0f : top;
          fa = ex2_approx_ftz(ref - safe);
          fb = ex2_approx_ftz(other - safe);
          l = l * fa + st.sum[r] * fb;
          ref = top;
        }
      }
      if (t == 0 || (x.step == 1 && shape.split == 1)) {
        const bool some = !(l == 0.0f);
        const bool whole = shape.split == 1;
        const float f = *dead ? NAN : !whole ? 1.0f : some ? 1.0f / l : 0.0f;
        fa *= f;
        fb *= f;
        const int64_t row = (int64_t)(x.q0 + token) * a.heads + x.kvh * a.group + head;
        if (whole) {
          if (there) a.lse[row] = *dead ? NAN : some ? (ref - C::LIFT + log2f(l)) * kLn2 : -INFINITY;
        } else {
          st.ref[r] = *dead ? NAN : ref;
          st.sum[r] = l;
        }
        const bool bad = *(volatile int32_t*)&st.bad != 0;
#pragma unroll 1
        for (int i = 0; i < C::DP; i += 32) {
          float o[32];
          if (mine > 0) {
            tc_load32(o_at + i, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= fa;
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = *dead ? NAN : 0.0f;
          }
          if (x.step == 2) {
            float q[32];
            tc_load32(o_at + C::DP + i, q);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = fmaf(q[j], fb, o[j]);
          }
          if (!some && !*dead) {  // no weight: 0, whatever O holds
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0.0f;
          }
          if (bad && there && i < a.d) {
            float again[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) again[j] = o[j];
            give_back<C::HALF>(a, x, lo, hi, i, again);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = again[j];
          }
          if (!whole) {  // for the cluster; every operand of the ring has been used
            if (there) {
              float* const share = reinterpret_cast<float*>(ring_ptr) + r * C::SHARE + i;
#pragma unroll
              for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(share + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
          } else if (there && i < a.d) {
            put_columns<C>(a, row, i, o);
          }
        }
      }
      tc_before();
      if (x.step == 2) {  // tile 1's O and sums have been read
        if (t == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(pair_empty);
        } else {
          wait_for(pair_empty, pairs & 1, dead);
        }
        ++pairs;
      }
    }
  }
  __syncwarp();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (*dead) {
    if (shape.split > 1) {
      if (threadIdx.x < 128) st.ref[threadIdx.x] = NAN;
    } else {
      for_last_items(st.work, [&](uint32_t id) {
        const Item x = item_of(a, shape, id, ids, 0, lane);
        const int vectors = a.d / 8;
#pragma unroll 1
        for (int i = threadIdx.x; i < (x.last - x.t0 + 1) * a.group * vectors; i += C::THREADS) {
          const int r = i / vectors;
          const int64_t row = (int64_t)(x.q0 + x.t0 + r / a.group) * a.heads + x.kvh * a.group + r % a.group;
          put_nan(a.out, row, vectors, i % vectors);
          if (a.rest) put_nan(a.rest, row, vectors, i % vectors);
          if (i % vectors == 0) a.lse[row] = NAN;
        }
      });
    }
  }
  if (shape.split > 1) {
    // The CTAs of the cluster join the rows that are there, eight columns a thread.
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const Item x = item_of(a, shape, first_id, ids, 0, lane);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int there = x.n0 >= 0 ? (x.last - x.t0 + 1) * a.group : 0, vectors = a.d / 8;
    const uint32_t refs = smem_at(st.ref), sums = smem_at(st.sum);
    auto at_rank = [&](uint32_t at, int rank) {
      uint32_t r;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
      return r;
    };
    auto remote = [&](uint32_t at, int rank) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at_rank(at, rank)));
      return v;
    };
#pragma unroll 1
    for (int u = part * C::THREADS + threadIdx.x; u < there * vectors; u += shape.split * C::THREADS) {
      const int r = u / vectors, col = (u - r * vectors) * 8;
      const uint32_t from = ring + (r * C::SHARE + col) * 4;
      float ref[8], sum[8], o[8], l = 0.0f, top = -INFINITY;
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        ref[z] = z < shape.split ? remote(refs + 4 * r, z) : -INFINITY;
        sum[z] = z < shape.split ? remote(sums + 4 * r, z) : 0.0f;
        o[z] = 0.0f;
        top = top != top || ref[z] <= top ? top : ref[z];  // NaN stays
      }
      const float safe = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        if (sum[z] == 0.0f) continue;  // no key, or no CTA
        const float f = ex2_approx_ftz(ref[z] - safe);
        l = fmaf(f, sum[z], l);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
                       : "r"(at_rank(from, z) + 4 * i));
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(v[i], f, o[i]);
      }
      if (top != top) l = NAN;  // a CTA that gave up
      const bool some = !(l == 0.0f);
      const float f = some ? 1.0f / l : 0.0f;
      const int64_t row = (int64_t)(x.q0 + x.t0 + r / a.group) * a.heads + x.kvh * a.group + r % a.group;
      if (col == 0) a.lse[row] = some ? (top - C::LIFT + log2f(l)) * kLn2 : -INFINITY;
      uint32_t w[4], low[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = some ? o[i] * f : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = pack16<C::HALF>(o[2 * i], o[2 * i + 1]);
        low[i] = pack16<C::HALF>(o[2 * i] - value16<C::HALF>((uint16_t)w[i]), o[2 * i + 1] - value16<C::HALF>((uint16_t)(w[i] >> 16)));
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.d + col) = make_uint4(w[0], w[1], w[2], w[3]);
      if (a.rest) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.rest) + row * a.d + col) = make_uint4(low[0], low[1], low[2], low[3]);
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <class C>
cudaError_t launch_fwd_of(const PromptArgs& a, cudaStream_t stream) {
  const int tp = 128 / a.group;
  auto items = [&](int tiles) { return ((int64_t)a.num_q / (tiles * tp) + a.nseq) * a.kv; };
  // One tile a CTA, on which both softmax groups work, where two would leave SMs without
  // any (as a graph, two tiles against one: 4 x 255 queries on 4354 keys, 16 heads over 2,
  // 57 us / 43; 1000 tokens 20.8 / 17.1; 2000 tokens, 252 items of one, 31.7 / 32.8). Then,
  // where SMs are to spare and each CTA keeps two blocks of keys, clusters (one CTA, 2, 4, 8:
  // a token over 8192 keys, 8 key heads, 64 us / 37 / 23 / 17, over 1024 13.6 / 11.9 / 10.1
  // / 10.0). More than 128 CTAs in clusters do not all reside (38 items of 300 queries on
  // 2300 keys: 26 / 22, and 33 with 152 CTAs; 32 of 8192 keys 66 / 39 / 29, and 50 with 256).
  FwdShape shape = {items(2) > 152 ? 2 : 1, 1};
  if (shape.tiles == 1) {
    int64_t keys = a.num_k / a.nseq;
    if (a.window && keys > (int64_t)a.window + tp) keys = (int64_t)a.window + tp;
    while (shape.split < 8 && items(1) * shape.split * 2 <= 128 && keys >= (int64_t)shape.split * 2 * 256) shape.split *= 2;
  }
  const int64_t blocks = items(shape.tiles) * shape.split;
  CUtensorMap mq, mk, mv;
  cudaError_t e = rows_map(&mq, a.q, C::HALF, a.d, a.heads, a.num_q, a.qt, a.qh, a.group, tp);
  if (e == cudaSuccess) e = rows_map(&mk, a.k, C::HALF, a.d, a.kv, a.num_k, a.kt, a.kh, 1, 128);
  if (e == cudaSuccess) e = rows_map(&mv, a.v, C::HALF, a.d, a.kv, a.num_k, a.vt, a.vh, 1, 128);
  auto* kernel = prompt_fwd_kernel<C>;
  if (e == cudaSuccess) e = allow_dynamic_smem((const void*)kernel, C::SMEM);
  if (e != cudaSuccess) return e;
  if (shape.split > 1)
    return launch_clusters(kernel, dim3((unsigned)blocks), dim3(C::THREADS), C::SMEM, (unsigned)shape.split, stream, a, shape, mq,
                           mk, mv);
  return launch_dependent(kernel, dim3((unsigned)blocks), dim3(C::THREADS), C::SMEM, stream, a, shape, mq, mk, mv);
}

template <int DP, bool WINDOW>
cudaError_t launch_fwd(const PromptArgs& a, bool half, cudaStream_t stream) {
  return half ? launch_fwd_of<Fwd<DP, true, WINDOW>>(a, stream) : launch_fwd_of<Fwd<DP, false, WINDOW>>(a, stream);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, bool half, cudaStream_t stream) {
  if (a.window) return a.d <= 64 ? launch_fwd<64, true>(a, half, stream) : launch_fwd<128, true>(a, half, stream);
  return a.d <= 64 ? launch_fwd<64, false>(a, half, stream) : launch_fwd<128, false>(a, half, stream);
}

}  // namespace csa
