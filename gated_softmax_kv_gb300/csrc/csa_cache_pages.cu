// Handling of the cache's pages (declared in include/csa_cache.h): copy,
// fork, reserve (allocation, copy on write), free, compact.
//
// Who gets which page is settled by one CTA per call with prefix sums over
// lists in memory, so the answer depends on the tables alone; the moving of
// page contents, the only part with real traffic, is a copy kernel over the
// whole GPU that reads how many pages there are to move from device memory,
// so no call waits for the host. Measured: reserve for 256 sequences 10 us, a
// chain of lookups and barriers; the plan of a compaction 8 us
// and the moving of 46 MB of pages 13.5 us (6.8 TB/s, the copy rate).
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_cache_internal.h"
#include "csa_device.cuh"

namespace csa {

namespace {

constexpr int kPlanThreads = 1024;

// Sum of v over the CTA's threads before this one; *total gets the whole sum.
template <typename T>
__device__ __forceinline__ T block_prefix(T v, T* total) {
  __shared__ T sums[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // sums may still be read by an earlier call
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    sums[lane] = w;
  }
  __syncthreads();
  *total = sums[kPlanThreads / 32 - 1];
  return x - v + (warp ? sums[warp - 1] : 0);
}

// ---- copying ------------------------------------------------------------------

struct CopyArgs {
  CacheView c;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;  // device word; null: n
  int32_t n;
  int32_t parts;         // pieces a page's data is cut into
};

constexpr int kPiece = 16384;  // bytes of a piece: 4 vectors a thread

__device__ __forceinline__ void copy_piece(const CacheView& c, int64_t src, int64_t dst, int part) {
  const int64_t bytes = ((int64_t)c.heads << c.page_bits) * c.d;
  const int64_t at = (int64_t)part * kPiece;
  const int vecs = (int)((bytes - at < kPiece ? bytes - at : kPiece) >> 4);
  const uint4* s = reinterpret_cast<const uint4*>(c.data + src * bytes + at);
  uint4* d = reinterpret_cast<uint4*>(c.data + dst * bytes + at);
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if ((int)threadIdx.x + 256 * k < vecs) v[k] = s[threadIdx.x + 256 * k];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if ((int)threadIdx.x + 256 * k < vecs) d[threadIdx.x + 256 * k] = v[k];
  if (part == 0) {
    const int64_t scales = (int64_t)c.heads << (c.page_bits - c.block_bits);
    for (int i = threadIdx.x; i < scales; i += 256)
      c.scales[dst * scales + i] = c.scales[src * scales + i];
  }
}

__device__ __forceinline__ void copy_pieces(const CopyArgs& a, int64_t first, int64_t stride) {
  const int64_t n = a.count ? *a.count : a.n;
  for (int64_t u = first; u < n * a.parts; u += stride) {
    const int64_t i = u / a.parts;
    const int32_t s = a.src[i], d = a.dst[i];
    if (s < 0 || d < 0 || s >= a.c.num_pages || d >= a.c.num_pages || s == d) continue;
    copy_piece(a.c, s, d, (int)(u - i * a.parts));
  }
}

__global__ void __launch_bounds__(256) copy_pages_kernel(const CopyArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  copy_pieces(a, blockIdx.x, gridDim.x);
}

int parts_of(const CacheView& c) {
  const int64_t bytes = ((int64_t)c.heads << c.page_bits) * c.d;
  return (int)((bytes + kPiece - 1) / kPiece);
}

unsigned copy_grid(int64_t pieces) {
  const int64_t most = 152 * 8;
  return (unsigned)(pieces < most ? pieces : most);
}

// ---- fork ---------------------------------------------------------------------

__device__ __forceinline__ bool test_and_set(uint32_t* bits, int i) {
  return (atomicOr(bits + (i >> 5), 1u << (i & 31)) >> (i & 31)) & 1;
}

__global__ void __launch_bounds__(kPlanThreads)
    fork_check_kernel(const int32_t* table, const int32_t* lens, int32_t nseq, int32_t max_pages,
                      int32_t page_bits, const int32_t* parents, const int32_t* children, int32_t n,
                      int32_t* status, int32_t* ok) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ uint32_t seen[];  // a bit a sequence
  __shared__ int found;
  for (int i = threadIdx.x; i < (nseq + 31) / 32; i += kPlanThreads) seen[i] = 0;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  int bits = 0;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int p = parents[i], c = children[i];
    if (p < 0 || p >= nseq || c < 0 || c >= nseq) {
      bits |= CSA_CACHE_BAD_SEQ;
      continue;
    }
    if (test_and_set(seen, c)) bits |= CSA_CACHE_DUPLICATE;
    if (lens[c] > 0 || table[(int64_t)c * max_pages] >= 0) bits |= CSA_CACHE_BUSY;
    if (lens[p] > ((int64_t)max_pages << page_bits)) bits |= CSA_CACHE_TABLE_FULL;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int p = parents[i];
    if (p >= 0 && p < nseq && ((seen[p >> 5] >> (p & 31)) & 1)) bits |= CSA_CACHE_DUPLICATE;
  }
  if (bits) atomicOr(&found, bits);
  __syncthreads();
  if (threadIdx.x == 0) {
    if (found) atomicOr(status, found);
    *ok = found == 0;
  }
}

__global__ void __launch_bounds__(256)
    fork_apply_kernel(int32_t* table, int32_t* lens, int32_t* refs, int32_t max_pages,
                      int32_t num_pages, int32_t page_bits, const int32_t* parents,
                      const int32_t* children, int32_t n, int32_t* status, const int32_t* ok) {
  grid_dependency_wait();
  allow_dependent_launch();
  if (!*ok) return;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t p = parents[i], c = children[i];
    const int len = max(lens[p], 0);
    const int held = (int)(((int64_t)len + (1 << page_bits) - 1) >> page_bits);
    for (int e = threadIdx.x; e < max_pages; e += 256) {
      const int page = e < held ? table[p * max_pages + e] : -1;
      table[c * max_pages + e] = page;
      if (page >= 0 && page < num_pages)
        atomicAdd(refs + page, 1);
      else if (e < held)
        atomicOr(status, CSA_CACHE_BAD_PAGE);
    }
    if (threadIdx.x == 0) lens[c] = len;
  }
}

// ---- reserve ------------------------------------------------------------------

struct ReserveArgs {
  CacheView c;
  int32_t* table;
  const int32_t* lens;
  int32_t* refs;
  int32_t nseq, max_pages;
  const int32_t* seqs;
  const int32_t* rows;
  int32_t n;
  int32_t* status;
  // workspace
  int32_t* need;   // [n] pages that request i takes, then their prefix sums
  int32_t* fresh;  // [num_pages] the pages taken, in order
  int32_t* asked;  // [num_pages] requests of this call that will write a shared page
  int32_t* last;   // [num_pages] 1 + the last of them
  int32_t* src;    // [num_pages] copies
  int32_t* dst;
  int32_t* count;
};

// Entries [lo, hi) of its table row that a request will write to.
struct Reach {
  int32_t s;
  int64_t lo, hi, len;
};
__device__ __forceinline__ Reach reach_of(const ReserveArgs& a, int i) {
  Reach r;
  r.s = a.seqs[i];
  const int64_t rows = a.rows[i];
  r.len = max(a.lens[r.s], 0);
  r.lo = r.len >> a.c.page_bits;
  r.hi = rows > 0 ? (r.len + rows + (1 << a.c.page_bits) - 1) >> a.c.page_bits : r.lo;
  return r;
}
constexpr int kShort = 4;  // entries that a thread goes through by itself

// Calls f(request, reach, first entry, stride, group) for every request: a
// thread by itself for a short one (a decoding step's: all of them at once), a
// warp for a long one. `group` is 1 or 32, the threads that share the request.
template <class F>
__device__ __forceinline__ void for_requests(const ReserveArgs& a, F f) {
  const int lane = threadIdx.x & 31;
  for (int i0 = (threadIdx.x >> 5) * 32; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + lane;
    Reach r = {0, 0, 0, 0};
    if (i < a.n) r = reach_of(a, i);
    const bool longer = r.hi - r.lo > kShort;
    if (i < a.n && !longer) f(i, r, r.lo, 1, 1);
    __syncwarp();
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, longer); left; left &= left - 1) {
      const int j = i0 + __ffs(left) - 1;
      const Reach q = reach_of(a, j);
      f(j, q, q.lo + lane, 32, 32);
      __syncwarp();
    }
  }
}

__device__ __forceinline__ bool in_pool(const ReserveArgs& a, int page) {
  return page >= 0 && page < a.c.num_pages;
}

// Whether request i replaces a held page: it is shared, and not left to it as
// the last of the requests that between them hold all of it.
__device__ __forceinline__ bool replaces(const ReserveArgs& a, int i, int page, int refs) {
  if (refs <= 1) return false;
  const int asked = *(volatile int32_t*)(a.asked + page);
  return refs > asked || *(volatile int32_t*)(a.last + page) != i + 1;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const ReserveArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ uint32_t seen[];
  __shared__ int found, copies;
  for (int i = threadIdx.x; i < (a.nseq + 31) / 32; i += kPlanThreads) seen[i] = 0;
  if (threadIdx.x == 0) {
    found = 0;
    copies = 0;
    *a.count = 0;
  }
  __syncthreads();
  int bits = 0;
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int s = a.seqs[i];
    if (s < 0 || s >= a.nseq) {
      bits |= CSA_CACHE_BAD_SEQ;
      continue;
    }
    if (test_and_set(seen, s)) bits |= CSA_CACHE_DUPLICATE;
    const int64_t end = (int64_t)max(a.lens[s], 0) + max(a.rows[i], 0);
    if (a.rows[i] > 0 && end > ((int64_t)a.max_pages << a.c.page_bits)) bits |= CSA_CACHE_TABLE_FULL;
  }
  if (bits) atomicOr(&found, bits);
  __syncthreads();
  if (found) {
    if (threadIdx.x == 0) atomicOr(a.status, found);
    return;
  }
  // requests that write each shared page: cleared, then counted
  for (int pass = 0; pass < 2; ++pass) {
    for_requests(a, [&](int i, const Reach& r, int64_t e, int step, int) {
      for (; e < r.hi; e += step) {
        const int page = a.table[(int64_t)r.s * a.max_pages + e];
        if (!in_pool(a, page) || a.refs[page] <= 1) continue;
        if (pass == 0) {
          a.asked[page] = 0;
          a.last[page] = 0;
        } else {
          atomicAdd(a.asked + page, 1);
          atomicMax(a.last + page, i + 1);
        }
      }
    });
    __syncthreads();
  }
  // pages that each request takes
  for_requests(a, [&](int i, const Reach& r, int64_t e, int step, int group) {
    int take = 0;
    for (; e < r.hi; e += step) {
      const int page = a.table[(int64_t)r.s * a.max_pages + e];
      if (page < 0)
        ++take;
      else if (!in_pool(a, page))
        bits |= CSA_CACHE_BAD_PAGE;
      else
        take += replaces(a, i, page, a.refs[page]);
    }
    if (group == 32) take = __reduce_add_sync(0xFFFFFFFFu, take);
    if (group == 1 || (threadIdx.x & 31) == 0) a.need[i] = take;
  });
  if (bits) atomicOr(a.status, bits);
  __syncthreads();
  int64_t wanted = 0;
  for (int b = 0; b < a.n; b += kPlanThreads) {
    const int i = b + threadIdx.x;
    int64_t total;
    const int64_t before = block_prefix(i < a.n ? (int64_t)a.need[i] : (int64_t)0, &total);
    // the prefix is used only if the whole sum fits the pool, hence 32 bits
    if (i < a.n) a.need[i] = (int)min(wanted + before, (int64_t)INT32_MAX);
    wanted += total;
  }
  // the lowest free pages
  int64_t got = 0;
  for (int b = 0; b < a.c.num_pages && got < wanted; b += 4 * kPlanThreads) {
    int free_[4], mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = b + 4 * threadIdx.x + k;
      free_[k] = p < a.c.num_pages && a.refs[p] == 0;
      mine += free_[k];
    }
    int total;
    int64_t at = got + block_prefix(mine, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (free_[k]) {
        if (at < wanted) a.fresh[at] = b + 4 * threadIdx.x + k;
        ++at;
      }
    got += total;
  }
  __syncthreads();
  if (got < wanted) {
    if (threadIdx.x == 0) atomicOr(a.status, CSA_CACHE_EXHAUSTED);
    return;
  }
  // Every request has to see the counts from before the call: the new table
  // entries and copies first, the counts after the barrier.
  for_requests(a, [&](int i, const Reach& r, int64_t e, int step, int group) {
    int at = a.need[i];
    const unsigned below = group == 32 ? (1u << (threadIdx.x & 31)) - 1 : 0;
    for (int64_t e0 = r.lo; e0 < r.hi; e0 += step, e += step) {
      int page = -1;
      bool take = false, shared = false;
      if (e < r.hi) {
        page = a.table[(int64_t)r.s * a.max_pages + e];
        shared = in_pool(a, page) && replaces(a, i, page, a.refs[page]);
        take = page < 0 || shared;
      }
      const unsigned takers = group == 32 ? __ballot_sync(0xFFFFFFFFu, take) : take;
      if (take) {
        const int got_page = a.fresh[at + __popc(takers & below)];
        a.table[(int64_t)r.s * a.max_pages + e] = got_page;
        if (shared) {
          // a page without rows is only replaced
          const int k = atomicAdd(&copies, 1);
          a.src[k] = page;
          a.dst[k] = (e << a.c.page_bits) < r.len ? got_page : page;
        }
      }
      at += __popc(takers);
    }
  });
  __syncthreads();
  for (int k = threadIdx.x; k < copies; k += kPlanThreads) atomicSub(a.refs + a.src[k], 1);
  for (int64_t k = threadIdx.x; k < wanted; k += kPlanThreads) a.refs[a.fresh[k]] = 1;
  if (threadIdx.x == 0) *a.count = copies;
}

// ---- free ---------------------------------------------------------------------

__global__ void __launch_bounds__(256)
    free_kernel(int32_t* table, int32_t* lens, int32_t* refs, int32_t nseq, int32_t max_pages,
                int32_t num_pages, const int32_t* seqs, int32_t n) {
  grid_dependency_wait();
  allow_dependent_launch();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = seqs[i];
    if (s < 0 || s >= nseq) continue;
    // an exchange hands each entry to one CTA, so a sequence listed twice
    // gives its pages back once
    for (int e = threadIdx.x; e < max_pages; e += 256) {
      const int page = atomicExch(table + (int64_t)s * max_pages + e, -1);
      if (page >= 0 && page < num_pages) atomicSub(refs + page, 1);
    }
    if (threadIdx.x == 0) lens[s] = 0;
  }
}

// ---- compact ------------------------------------------------------------------

__global__ void __launch_bounds__(kPlanThreads)
    compact_kernel(int32_t* refs, int32_t pages, int32_t* src, int32_t* dst, int32_t* map,
                   int32_t* count, int32_t* limit, int32_t* live) {
  grid_dependency_wait();
  allow_dependent_launch();
  int held = 0;
  for (int p = threadIdx.x; p < pages; p += kPlanThreads) held += refs[p] > 0;
  int L;
  block_prefix(held, &L);
  // holes below L and held pages from L on are equally many
  int holes = 0, movers = 0;
  for (int b = 0; b < pages; b += 4 * kPlanThreads) {
    int kind[4], h = 0, m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = b + 4 * threadIdx.x + k;
      kind[k] = 0;
      if (p < pages) {
        const bool used = refs[p] > 0;
        if (p < L && !used) kind[k] = 1;
        if (p >= L && used) kind[k] = 2;
        if (p >= L && !used) map[p] = p;
      }
      h += kind[k] == 1;
      m += kind[k] == 2;
    }
    int th, tm;
    int ah = holes + block_prefix(h, &th);
    int am = movers + block_prefix(m, &tm);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = b + 4 * threadIdx.x + k;
      if (kind[k] == 1) dst[ah++] = p;
      if (kind[k] == 2) src[am++] = p;
    }
    holes += th;
    movers += tm;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlanThreads) {
    const int s = src[i], d = dst[i];
    map[s] = d;
    refs[d] = refs[s];
    refs[s] = 0;
  }
  if (threadIdx.x == 0) {
    *count = movers;
    *limit = L;
    if (live) *live = L;
  }
}

__global__ void __launch_bounds__(256)
    compact_move_kernel(const CopyArgs a, int32_t* table, int64_t entries, const int32_t* map,
                        const int32_t* limit) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int L = *limit;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries;
       i += (int64_t)gridDim.x * 256) {
    const int p = table[i];
    if (p >= L && p < a.c.num_pages) table[i] = map[p];
  }
  copy_pieces(a, blockIdx.x, gridDim.x);
}

csa_status_t done(cudaError_t e) { return e == cudaSuccess ? CSA_OK : record_cuda_error(e); }

// The table, lengths and counts that every call here takes.
csa_status_t check_tables(const void* table, const void* lens, const void* refs, int32_t num_seqs,
                          int32_t max_pages, int32_t num_pages) {
  if (num_seqs < 1 || num_seqs > kMaxSeqs || max_pages < 1 || max_pages > kMaxPages ||
      num_pages < 1 || num_pages > (1 << 24))
    return CSA_ERR_RANGE;
  if (!table || !lens || !refs) return CSA_ERR_NULL;
  if (misaligned4(table) || misaligned4(lens) || misaligned4(refs)) return CSA_ERR_ALIGN;
  return CSA_OK;
}

csa_status_t check_list(const void* a, const void* b, int32_t n, int32_t most) {
  if (n < 0 || n > most) return CSA_ERR_RANGE;
  if (n > 0 && (!a || !b)) return CSA_ERR_NULL;
  if (misaligned4(a) || misaligned4(b)) return CSA_ERR_ALIGN;
  return CSA_OK;
}

}  // namespace

}  // namespace csa

extern "C" {

csa_status_t csa_cache_copy_pages(const csa_cache_t* cache, const int32_t* src, const int32_t* dst,
                                  int32_t n, cudaStream_t stream) {
  csa_status_t st = csa::check_cache(cache);
  if (st == CSA_OK) st = csa::check_list(src, dst, n, INT32_MAX);
  if (st != CSA_OK || n == 0) return st;
  csa::CopyArgs a;
  a.c = csa::view_of(cache);
  a.src = src;
  a.dst = dst;
  a.count = nullptr;
  a.n = n;
  a.parts = csa::parts_of(a.c);
  return csa::done(csa::launch_dependent(csa::copy_pages_kernel,
                                         dim3(csa::copy_grid((int64_t)n * a.parts)), dim3(256), 0,
                                         stream, a));
}

csa_status_t csa_cache_fork(int32_t* page_table, int32_t* seq_lens, int32_t* page_refs,
                            int32_t num_seqs, int32_t max_pages, int32_t num_pages,
                            int32_t page_size, const int32_t* parents, const int32_t* children,
                            int32_t n, int32_t* status, cudaStream_t stream) {
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return CSA_ERR_UNSUPPORTED;
  csa_status_t st =
      csa::check_tables(page_table, seq_lens, page_refs, num_seqs, max_pages, num_pages);
  if (st == CSA_OK) st = csa::check_list(parents, children, n, csa::kMaxSeqs);
  if (st != CSA_OK) return st;
  if (!status) return CSA_ERR_NULL;
  if (csa::misaligned4(status)) return CSA_ERR_ALIGN;
  if (n == 0) return CSA_OK;
  const int bits = csa::log2_of(page_size);
  void* ws = nullptr;
  cudaError_t e = csa::workspace_take(&ws, 16, stream);
  if (e != cudaSuccess) return csa::record_cuda_error(e);
  int32_t* ok = static_cast<int32_t*>(ws);
  const size_t smem = ((size_t)num_seqs + 31) / 32 * 4;
  e = csa::launch_dependent(csa::fork_check_kernel, dim3(1), dim3(csa::kPlanThreads), smem, stream,
                            (const int32_t*)page_table, (const int32_t*)seq_lens, num_seqs,
                            max_pages, bits, parents, children, n, status, ok);
  if (e == cudaSuccess)
    e = csa::launch_dependent(csa::fork_apply_kernel, dim3((unsigned)(n < 1216 ? n : 1216)),
                              dim3(256), 0, stream, page_table, seq_lens, page_refs, max_pages,
                              num_pages, bits, parents, children, n, status, (const int32_t*)ok);
  const cudaError_t ef = csa::workspace_give(ws, stream);
  return csa::done(e != cudaSuccess ? e : ef);
}

csa_status_t csa_cache_reserve(const csa_cache_t* cache, int32_t* page_table,
                               const int32_t* seq_lens, int32_t* page_refs, int32_t num_seqs,
                               int32_t max_pages, const int32_t* seqs, const int32_t* rows,
                               int32_t n, int32_t* status, cudaStream_t stream) {
  csa_status_t st = csa::check_cache(cache);
  if (st == CSA_OK)
    st = csa::check_tables(page_table, seq_lens, page_refs, num_seqs, max_pages, cache->num_pages);
  if (st == CSA_OK) st = csa::check_list(seqs, rows, n, csa::kMaxSeqs);
  if (st != CSA_OK) return st;
  if (!status) return CSA_ERR_NULL;
  if (csa::misaligned4(status)) return CSA_ERR_ALIGN;
  if (n == 0) return CSA_OK;
  csa::ReserveArgs a;
  a.c = csa::view_of(cache);
  a.table = page_table;
  a.lens = seq_lens;
  a.refs = page_refs;
  a.nseq = num_seqs;
  a.max_pages = max_pages;
  a.seqs = seqs;
  a.rows = rows;
  a.n = n;
  a.status = status;
  const int64_t pages = cache->num_pages;
  void* ws = nullptr;
  cudaError_t e = csa::workspace_take(&ws, 4 * (size_t)((int64_t)n + 5 * pages + 1), stream);
  if (e != cudaSuccess) return csa::record_cuda_error(e);
  int32_t* w = static_cast<int32_t*>(ws);
  a.need = w;
  a.fresh = w + n;
  a.asked = a.fresh + pages;
  a.last = a.asked + pages;
  a.src = a.last + pages;
  a.dst = a.src + pages;
  a.count = a.dst + pages;
  const size_t smem = ((size_t)num_seqs + 31) / 32 * 4;
  e = csa::launch_dependent(csa::reserve_kernel, dim3(1), dim3(csa::kPlanThreads), smem, stream, a);
  if (e == cudaSuccess) {
    csa::CopyArgs c;
    c.c = a.c;
    c.src = a.src;
    c.dst = a.dst;
    c.count = a.count;
    c.n = 0;
    c.parts = csa::parts_of(a.c);
    e = csa::launch_dependent(csa::copy_pages_kernel,
                              dim3(csa::copy_grid((n < pages ? n : pages) * c.parts)), dim3(256), 0,
                              stream, c);
  }
  const cudaError_t ef = csa::workspace_give(ws, stream);
  return csa::done(e != cudaSuccess ? e : ef);
}

csa_status_t csa_cache_free(int32_t* page_table, int32_t* seq_lens, int32_t* page_refs,
                            int32_t num_seqs, int32_t max_pages, int32_t num_pages,
                            const int32_t* seqs, int32_t n, cudaStream_t stream) {
  csa_status_t st =
      csa::check_tables(page_table, seq_lens, page_refs, num_seqs, max_pages, num_pages);
  if (st == CSA_OK) st = csa::check_list(seqs, seqs, n, csa::kMaxSeqs);
  if (st != CSA_OK || n == 0) return st;
  return csa::done(csa::launch_dependent(
      csa::free_kernel, dim3((unsigned)(n < 1216 ? n : 1216)), dim3(256), 0, stream, page_table,
      seq_lens, page_refs, num_seqs, max_pages, num_pages, seqs, n));
}

csa_status_t csa_cache_compact(const csa_cache_t* cache, int32_t* page_table, int32_t* page_refs,
                               int32_t num_seqs, int32_t max_pages, int32_t* live,
                               cudaStream_t stream) {
  csa_status_t st = csa::check_cache(cache);
  if (st == CSA_OK)
    st = csa::check_tables(page_table, page_table, page_refs, num_seqs, max_pages,
                           cache->num_pages);
  if (st != CSA_OK) return st;
  if (csa::misaligned4(live)) return CSA_ERR_ALIGN;
  const int64_t pages = cache->num_pages;
  void* ws = nullptr;
  cudaError_t e = csa::workspace_take(&ws, 4 * (size_t)(3 * pages + 2), stream);
  if (e != cudaSuccess) return csa::record_cuda_error(e);
  int32_t* src = static_cast<int32_t*>(ws);
  int32_t *dst = src + pages, *map = dst + pages, *count = map + pages, *limit = count + 1;
  e = csa::launch_dependent(csa::compact_kernel, dim3(1), dim3(csa::kPlanThreads), 0, stream,
                            page_refs, (int32_t)pages, src, dst, map, count, limit, live);
  if (e == cudaSuccess) {
    csa::CopyArgs c;
    c.c = csa::view_of(cache);
    c.src = src;
    c.dst = dst;
    c.count = count;
    c.n = 0;
    c.parts = csa::parts_of(c.c);
    const int64_t entries = (int64_t)num_seqs * max_pages;
    const int64_t rewrites = (entries + 255) / 256, moves = pages * c.parts;
    e = csa::launch_dependent(csa::compact_move_kernel,
                              dim3(csa::copy_grid(moves > rewrites ? moves : rewrites)), dim3(256),
                              0, stream, c, page_table, entries, (const int32_t*)map,
                              (const int32_t*)limit);
  }
  const cudaError_t ef = csa::workspace_give(ws, stream);
  return csa::done(e != cudaSuccess ? e : ef);
}

}  // extern "C"
