// How the attention's work is dealt out. An item is one tile of query rows of
// one (sequence, cache head); its keys are cut into chunks. All chunks of all
// items, in order, are one line of `total` units that the workers (CTAs) share
// in equal stretches, so ragged lengths balance without a plan made on the
// host. An item that lies across a stretch's end is finished by a second
// kernel from the workers' partial results, in the workers' order. The
// stretches depend on the lengths and sizes of the call alone.
#pragma once

#include <stdint.h>

#include "csa_cache_attend.h"

namespace csa {

struct PlanShape {
  int32_t row_bits;  // log2 of the query rows of a tile
  int32_t key_bits;  // log2 of the keys of a chunk
  int32_t workers;
  int32_t least;     // fewest chunks a worker takes
  bool whole;        // items are not cut: one unit each
  int32_t split;     // thread blocks of a cluster, which is then a worker (whole items)
};

struct SeqWork {
  int64_t tiles, chunks;  // tiles of a cache head; chunks of a tile
  int64_t keys;           // rows that the sequence holds and the table reaches
};

__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, const PlanShape& p, int s) {
  // no more queries than the call has, whatever cu holds: the line stays finite
  const int64_t nq = min((int64_t)__ldg(a.cu + s + 1), a.tokens) - max((int64_t)__ldg(a.cu + s), (int64_t)0);
  SeqWork w;
  w.keys = __ldg(a.lens + s);
  const int64_t most = (int64_t)a.max_pages << a.c.page_bits;
  if (w.keys > most) w.keys = most;
  if (w.keys < 0) w.keys = 0;
  w.tiles = nq > 0 ? (nq * a.group + (1 << p.row_bits) - 1) >> p.row_bits : 0;
  w.chunks = w.keys > 0 && !p.whole ? (w.keys + (1 << p.key_bits) - 1) >> p.key_bits : 1;
  return w;
}

struct Place {
  int64_t per;     // chunks of a stretch
  int64_t pos;     // first chunk of the stretch (-1: behind the end)
  int64_t end;     // chunk behind the stretch
  int64_t within;  // pos counted from the sequence's first chunk
  int32_t s;       // sequence that pos lies in
};

// Finds worker w's stretch; every thread of the CTA (THREADS of them) calls it
// and gets the answer. `sums` is shared memory for THREADS / 32 + 1 sums.
template <int THREADS>
__device__ __forceinline__ Place locate(const AttendArgs& a, const PlanShape& p, int64_t w,
                                        int64_t* sums, Place* found) {
  const int each = (a.nseq + THREADS - 1) / THREADS;
  const int s0 = min((int)threadIdx.x * each, a.nseq), s1 = min(s0 + each, a.nseq);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    const SeqWork k = seq_work(a, p, s);
    mine += k.tiles * k.chunks * a.kv;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  if (threadIdx.x == 0) found->pos = -1;
  __syncthreads();
  int64_t before = x - mine, total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += sums[i];
    total += sums[i];
  }
  int64_t per = (total + p.workers - 1) / p.workers;
  if (per < p.least) per = p.least;
  const int64_t pos = w * per;
  if (pos < total && pos >= before && pos < before + mine) {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      const SeqWork k = seq_work(a, p, s);
      const int64_t n = k.tiles * k.chunks * a.kv;
      if (pos < at + n) {
        found->per = per;
        found->pos = pos;
        found->end = min(pos + per, total);
        found->within = pos - at;
        found->s = s;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return *found;
}

// The plan of a call, on the host. Items of at most `few` chunks, as the table's
// width shows, are not worth cutting: no workspace, no joining kernel, and as
// many workers as there can be items, up to four for each that is resident (300
// rows by 16 heads: 20 us a call, cut and joined 26).
// Where so few items leave SMs free, the blocks of a cluster share an item's
// keys, `groups` chunks a block at a time (0: the kernel has no clusters): the same
// rows take 13.9 us by 8 blocks, 21.5 by one. A step is 2 us; four cost no more
// than the second kernel (5 us) and its workspace.
inline PlanShape plan_of(const AttendArgs& a, int rows, int keys, int resident, int least, int few, int groups) {
  PlanShape p;
  p.row_bits = log2_of(rows);
  p.key_bits = log2_of(keys);
  p.least = least;
  p.workers = resident;
  const int64_t chunks = (((int64_t)a.max_pages << a.c.page_bits) + keys - 1) / keys;
  const int64_t items = ((a.tokens * a.group) / rows + a.nseq) * a.kv;
  p.split = 1;
  while (p.split < 8 && groups > 0 && items * p.split * 2 <= 152 && chunks > p.split * groups) p.split *= 2;
  p.whole = chunks <= few || (p.split > 1 && chunks <= 4 * p.split * groups);
  if (!p.whole) p.split = 1;
  if (p.whole) {
    p.workers = (int32_t)(items < 4 * resident ? items : 4 * resident);
    p.least = 1;
  }
  return p;
}

}  // namespace csa
