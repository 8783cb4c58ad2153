// Shared by the tcgen05 kernels of causal attention over packed sequences: tiles of
// query rows, what they see, and cleaning of operands. Not installed.
//
// A tile is 128 rows of the matrix instructions: `tp` tokens by the `group` query
// heads of a key head (row = token * group + head), so that heads that share keys
// share a tile whatever their number, and the keys are read once for all of them.
// tp = 128 / group; rows at or behind tp * group are not used.
//
// Which tile is whose: slot(s) = floor(cu[s] / B) + s is the first slot of sequence
// s for stretches of B tokens, since ceil(n / B) <= floor((c + n) / B) - floor(c / B)
// + 1. So a CTA finds its sequence by searching cu, with no prefix sums and at most
// one slot a sequence that has no work.
#pragma once

#include <cuda_fp16.h>

#include "csa_device.cuh"
#include "csa_prompt_internal.h"
#include "csa_tc.cuh"

namespace csa {

__device__ __forceinline__ int64_t first_slot(const int32_t* cu, int s, int b) {
  return (int64_t)(max(__ldg(cu + s), 0) / b) + s;
}

// The last s in [0, nseq) whose first slot is at or before `slot`, by a warp, 32 at
// a time.
__device__ __forceinline__ int seq_of_slot(const int32_t* cu, int nseq, int b, int64_t slot, int lane) {
  int lo = 0, span = nseq;
  while (span > 1) {
    const int step = (span + 31) / 32, at = lo + lane * step;
    const bool before = lane * step < span && first_slot(cu, at, b) <= slot;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, before);
    const int k = who ? 31 - __clz(who) : 0;
    span = min(step, span - k * step);
    lo += k * step;
  }
  return lo;
}

// Rows of no sequence: [0, cu[0]) and [cu[nseq], n), a thread's share (every `step`-th
// from `from` on) of `words` 16-byte vectors of zeros a row.
__device__ __forceinline__ void fill_rest(const int32_t* cu, int nseq, int32_t n, int64_t words, uint4* to, int64_t from,
                                          int64_t step) {
  const int64_t a = min(max(__ldg(cu), 0), n), b = max((int64_t)min(max(__ldg(cu + nseq), 0), n), a);
#pragma unroll 1
  for (int64_t i = from; i < (a + n - b) * words; i += step) {
    const int64_t row = i / words;
    to[row < a ? i : i + (b - a) * words] = make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void fill_rest(const int32_t* cu, int nseq, int32_t n, int32_t heads, float v, float* to,
                                          int64_t from, int64_t step) {
  const int64_t a = min(max(__ldg(cu), 0), n), b = max((int64_t)min(max(__ldg(cu + nseq), 0), n), a);
#pragma unroll 1
  for (int64_t i = from; i < (a + n - b) * heads; i += step)
    to[i / heads < a ? i : i + (b - a) * heads] = v;
}

// ---- waits --------------------------------------------------------------------
//
// Bounded: `polls` of them without the phase mark the CTA, and no further wait waits. A CTA
// that gave up copies and takes over nothing more, waits for what it has under way (`land`),
// and writes NaN over the results of its last items (ids). A poll that fails takes about 2700
// cycles (1.4 us), so the usual kPolls of them 1.4 s, for what takes microseconds: a copy, a
// product, a tile's arithmetic.
struct Dead {
  volatile int32_t* flag;
  int32_t polls;
  __device__ __forceinline__ volatile int32_t& operator*() const { return *flag; }
};

// In this form, a hundred times inlined: with the limit tested before the first poll, or held in
// shared memory, 12 ragged sequences take 164 to 166 us instead of 159, 16384 tokens 710 to
// 717 instead of 697.
__device__ __forceinline__ void wait_for(uint32_t bar, uint32_t parity, const Dead& dead) {
  int i = 0;
#pragma unroll 1
  do {
    if (mbar_try(bar, parity)) return;
    if (*dead) return;
  } while (++i < dead.polls);
  *dead = 1;
}

// Whether the CTA has given up, the same for a whole warp.
__device__ __forceinline__ bool gave_up(const Dead& dead) { return __any_sync(0xFFFFFFFFu, *dead != 0); }

// For what may take as long as an item, and that is as long as the sequence: as many polls
// each time that *progress (a count of tiles) has moved since the last.
__device__ __forceinline__ void wait_through(uint32_t bar, uint32_t parity, const Dead& dead, const volatile uint32_t* progress) {
  uint32_t seen = *progress;
#pragma unroll 1
  for (int i = 0; !mbar_try(bar, parity); ++i) {
    if (*dead) return;
    if (i < dead.polls) continue;
    const uint32_t now = *progress;
    if (now == seen) {
      *dead = 1;
      return;
    }
    seen = now;
    i = 0;
  }
}

// For what the hardware has under way, copies, products or an answer, which ends by itself
// and before the CTA may.
__device__ __forceinline__ bool land(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < kPolls; ++i)
    if (mbar_try(bar, parity)) return true;
  return false;
}
// The last `stages` of a ring's copies.
__device__ __forceinline__ void land_ring(uint32_t full, uint32_t stages, uint32_t issued) {
#pragma unroll 1
  for (uint32_t j = issued > stages ? issued - stages : 0; j < issued; ++j) land(full + 8 * (j % stages), (j / stages) & 1);
}

// ---- items of work -----------------------------------------------------------
//
// A warp of its own finds the items (type Item, n0 < 0: none): first the CTA's own, then
// those of CTAs that have not started and are cancelled for it (cluster launch control),
// until there are none. It looks for the next one when the warp of the matrix
// instructions says that the last is near its end (want_work), no earlier: an item
// taken at once would wait behind a long one while other SMs run dry (4096 tokens, 32
// heads of 128, dK and dV: 254 us instead of 197).

struct WorkState {
  alignas(16) uint32_t stolen[4];
  uint64_t full[2], empty[2], steal, want, ended;  // ended: the products
  uint32_t progress;  // tiles that the cleaning warp has seen
  // Of the items that were found, by their number: unfinished are at most the one whose
  // result is formed, two in the slots and one that waits for a slot.
  uint32_t ids[4];
  int32_t found;
};

__device__ __forceinline__ void init_work(WorkState& w, int takers) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(smem_at(&w.full[i]), 1);
    mbar_init(smem_at(&w.empty[i]), takers);
  }
  mbar_init(smem_at(&w.steal), 1);
  mbar_init(smem_at(&w.want), 1);
  mbar_init(smem_at(&w.ended), 1);
  w.progress = 0;
  w.found = 0;
}

template <class Item, class Find>
__device__ __forceinline__ void find_work(WorkState& w, Item* slots, uint32_t id, bool once, int lane, const Dead& dead,
                                          Find find) {
  const uint32_t full = smem_at(w.full), empty = smem_at(w.empty), steal = smem_at(&w.steal), stolen = smem_at(w.stolen);
  int k = 0;
  uint32_t wanted = 0;
#pragma unroll 1
  for (int n = 0;; ++n) {
    const Item x = find(id);
    if (x.n0 >= 0) {
      if (lane == 0) {
        w.ids[k & 3] = id;
        w.found = k + 1;
      }
      wait_for(empty + 8 * (k & 1), ((k >> 1) & 1) ^ 1, dead);
      if (gave_up(dead)) return;  // the slot may be in use, and no one takes it any more
      if (lane == 0) {
        slots[k & 1] = x;
        mbar_arrive(full + 8 * (k & 1));
      }
      ++k;
    }
    if (once) break;
    if (x.keys()) wait_through(smem_at(&w.want), wanted++ & 1, dead, &w.progress);
    if (gave_up(dead)) return;
    if (lane == 0) {
      mbar_expect(steal, 16);
      asm volatile(
          "fence.proxy.async.shared::cta;\n\t"
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(stolen),
          "r"(steal)
          : "memory");
    }
    if (!__any_sync(0xFFFFFFFFu, land(steal, n & 1))) {
      *dead = 1;
      return;
    }
    uint32_t got;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(id)
        : "r"(stolen)
        : "memory");
    if (!got) break;
  }
  wait_for(empty + 8 * (k & 1), ((k >> 1) & 1) ^ 1, dead);
  if (gave_up(dead)) return;
  if (lane == 0) {
    slots[k & 1].n0 = -1;
    mbar_arrive(full + 8 * (k & 1));
  }
}

// Work goes on: the cleaning warp, which has time, once a tile of the ring (in the warp of the
// matrix instructions it costs 16384 tokens 6 us of 700).
__device__ __forceinline__ void tile_seen(WorkState& w, int lane) {
  if (lane == 0) *(volatile uint32_t*)&w.progress = w.progress + 1;
}

// The warp of the matrix instructions, when it has issued its last: the products are done.
__device__ __forceinline__ void end_products(WorkState& w, uint32_t leader) {
  tc_commit_by(leader, smem_at(&w.ended));
  land(smem_at(&w.ended), 0);
}

// For a CTA that gave up, when its warps have met: f(id) for its last items.
template <class F>
__device__ __forceinline__ void for_last_items(const WorkState& w, F f) {
#pragma unroll 1
  for (int k = max(0, w.found - 4); k < w.found; ++k) f(w.ids[k & 3]);
}
// NaN of either type in a row of `vectors` 16-byte vectors.
__device__ __forceinline__ void put_nan(void* to, int64_t row, int vectors, int at) {
  static_cast<uint4*>(to)[row * vectors + at] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
}

// Once for each item with work for the matrix instructions (Item::keys).
__device__ __forceinline__ void want_work(WorkState& w, int lane) {
  if (lane == 0) mbar_arrive(smem_at(&w.want));
}

// The k-th item, for a whole warp; its slot may be filled again after that.
template <class Item>
__device__ __forceinline__ Item take_work(WorkState& w, const Item* slots, int k, int lane, const Dead& dead) {
  wait_for(smem_at(&w.full[k & 1]), (k >> 1) & 1, dead);
  Item x = slots[k & 1];
  if (gave_up(dead)) x.n0 = -1;
  if (lane == 0) mbar_arrive(smem_at(&w.empty[k & 1]));
  return x;
}

// A place in the ring, and the parity of its barriers.
template <int NS>
struct Place {
  int stage;
  uint32_t parity;
  __device__ __forceinline__ void next(int n) {
    stage += n;
    if (stage >= NS) {
      stage -= NS;
      parity ^= 1;
    }
  }
};

// Half a word pair whose exponent is all ones: infinity or NaN.
template <bool HALF>
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {
  constexpr uint32_t E = HALF ? 0x7C00u : 0x7F80u;
  uint32_t keep = 0;
  if ((w & E) != E) keep |= 0xFFFFu;
  if ((w & (E << 16)) != (E << 16)) keep |= 0xFFFF0000u;
  return keep;
}
// Whether some half of the words does: an exponent of ones carries into the half's
// sign bit, which has been cleared.
template <bool HALF>
__device__ __forceinline__ uint32_t infinite_bits(uint4 v) {
  constexpr uint32_t E = HALF ? 0x7C007C00u : 0x7F807F80u, ONE = HALF ? 0x04000400u : 0x00800080u;
  return (((v.x & E) + ONE) | ((v.y & E) + ONE) | ((v.z & E) + ONE) | ((v.w & E) + ONE)) & 0x80008000u;
}

// Zeros for infinities and NaN in `bytes` (a multiple of 4096) of an operand in shared
// memory, by a warp; *found is set where there were any. A weight of 0 keeps a finite
// value out of a sum, but not these. A warp of its own does this ahead of the products: as
// a part of the softmax it cost 3600 cycles a block (5003 tokens of 64 heads of 64 with a
// window of 128: 140 us).
template <bool HALF>
__device__ __forceinline__ void clean_operand(uint8_t* at, int bytes, int lane, volatile int32_t* found) {
  bool any = false;
#pragma unroll 1
  for (int i = lane * 16; i < bytes; i += 4096) {
    uint4 v[8];
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const uint4*>(at + i + k * 512);
#pragma unroll
    for (int k = 0; k < 8; ++k) bits |= infinite_bits<HALF>(v[k]);
    if (bits) {
      *found = 1;
      any = true;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4*>(at + i + k * 512) =
            make_uint4(v[k].x & finite_mask<HALF>(v[k].x), v[k].y & finite_mask<HALF>(v[k].y), v[k].z & finite_mask<HALF>(v[k].z),
                       v[k].w & finite_mask<HALF>(v[k].w));
    }
  }
  if (__any_sync(0xFFFFFFFFu, any)) fence_async();
}

template <bool HALF>
__device__ __forceinline__ float value16(uint16_t b) {
  return HALF ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (HALF) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return pack_bf16x2(lo, hi);
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 32 bytes, a sector, at once.
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A tensor map of [tokens, heads, d] rows: boxes of 64 columns, `heads_box` heads and
// `tokens_box` tokens. (csa_prompt.cu)
cudaError_t rows_map(CUtensorMap* map, const void* base, bool half, int32_t d, int32_t heads, int64_t tokens, int64_t ts,
                     int64_t hs, int32_t heads_box, int32_t tokens_box);

}  // namespace csa
