/*
 * csa_cache.h -- C ABI of the paged 8-bit cache of compressed rows, the
 * attention that reads it and the handling of its pages (part of
 * libcsa_compress.so).
 *
 * The cache is a pool of pages. A page holds page_size rows of num_heads
 * heads of head_dim columns in e4m3 (8-bit floating point: sign, four
 * exponent and three mantissa bits; largest finite value 448, one NaN, no
 * infinity), and one fp32 scale for every `block` consecutive rows of a head:
 *
 *   data    e4m3 [num_pages, num_heads, page_size, head_dim]
 *   scales  fp32 [num_pages, num_heads, page_size / block]
 *
 * and stands for the values data * scale. Sequence s holds seq_lens[s] rows;
 * row j lies in slot j % page_size of page page_table[s, j / page_size]
 * (int32 [num_seqs, max_pages]; -1: no page).
 *
 * Scales that csa_cache_append writes are powers of two. A value's rounding
 * to e4m3 is relative, so a power of two loses nothing against amax / 448
 * but the range below 2^-6 of the scale; in return the values the cache
 * stands for are exact in fp16 and bf16 (up to their exponent range), and a
 * block whose scale grows is requantised without a second rounding of its
 * normal values. csa_cache_attend takes any finite scales >= 0.
 *
 * All pointers are caller-owned device memory on the current device;
 * nothing is retained. Calls are asynchronous on `stream`, never synchronise
 * the host, can be captured into a graph, and validate sizes, alignment and
 * null pointers on the host before any launch (CSA_ERR_*). Tables, lengths and
 * index lists are read on the device only. Kernels stay inside the buffers
 * whatever those hold: a page outside [0, num_pages) or a row outside the
 * table is treated as not there (not read, not written, not seen). max_pages
 * is at most 2^27, num_seqs and the lists of sequences at most 262144 long.
 */
#ifndef CSA_CACHE_H
#define CSA_CACHE_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "csa_compress.h"
#include "csa_rope.h" /* CSA_BF16, CSA_FP16, CSA_FP32 */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Envelope: head_dim in {64, 128, 256, 512}; page_size in {16, 32, 64, 128,
 * 256}; block a power of two <= page_size; num_heads in 1 .. 1024; num_pages
 * 1 .. 2^24. data 16-byte aligned, scales 4-byte aligned. Flat offsets are 64
 * bits wide.
 */
typedef struct csa_cache {
  void* data;
  float* scales;
  int32_t num_pages;
  int32_t num_heads;
  int32_t page_size;
  int32_t block;
  int32_t head_dim;
} csa_cache_t;

/*
 * Appends rows: sequence s gets rows cu_rows[s] .. cu_rows[s + 1] - 1 of
 * `rows` [num_rows, num_heads, head_dim] (dtype CSA_BF16, CSA_FP16 or
 * CSA_FP32; last dimension contiguous, row and head strides in elements,
 * multiples of 16 bytes) as its rows seq_lens[s], seq_lens[s] + 1, ... The
 * pages must be there (csa_cache_reserve) and be held by no other sequence;
 * seq_lens is read, not changed (the caller adds the lengths afterwards).
 * rows at or behind cu_rows[num_seqs] are not read.
 *
 * For each (block, head) that gets rows, the new scale is the smallest power
 * of two 2^k >= amax / 448 over the new rows' finite values, k in [-120,
 * 120], or the block's old scale if that is larger and the block already held
 * rows of this sequence, which are requantised when the scale grew. Values
 * are rounded to nearest even; infinities and NaN are stored as NaN. Slots of
 * the block behind the last row keep what they hold. Appending row by row
 * gives the bits of appending at once, except for values that fall below 2^-6
 * of the final scale, which may have been rounded twice.
 * One launch; num_rows == 0 launches nothing. (num_rows / block + 2 num_seqs) *
 * num_heads < 2^31.
 */
csa_status_t csa_cache_append(const csa_cache_t* cache, const void* rows, int32_t dtype,
                              int64_t num_rows, int64_t row_stride, int64_t head_stride,
                              const int32_t* page_table, int32_t num_seqs, int32_t max_pages,
                              const int32_t* seq_lens, const int32_t* cu_rows,
                              cudaStream_t stream);

/*
 * Attention of packed queries over the cache. Sequence s has the query tokens
 * cu_q[s] .. cu_q[s + 1] - 1 of q [num_tokens, num_q_heads, head_dim] (dtype
 * CSA_BF16 or CSA_FP16; last dimension contiguous, strides in elements,
 * multiples of 16 bytes). Query head h reads cache head h / (num_q_heads /
 * kv_heads) as its keys and, with `shared`, the same rows as its values (one
 * latent row a token for key and value), else cache head kv_heads + that one:
 *
 *   z_j = sm_scale * (q . key_j)   for rows j < min(visible[t], seq_lens[s])
 *   out = sum_j softmax(z)_j value_j          lse = log sum_j exp(z_j)
 *
 * visible [num_tokens] (int32) may be null: every row of the sequence is
 * seen. A compressed row that ends at token (j + 1) * ratio - 1 is in the
 * past of the query at position p when j < (p + 1) / ratio. Rows that a query
 * does not see take no part in its sums, whatever they and their scales hold
 * (NaN and infinities included). Only roundings can differ: queries that are
 * worked on together rescale their sums at the same rows.
 * A query that sees no row, or whose logits are all -inf (those below -6e37
 * count as -inf), gets out 0 and lse -inf. out [num_tokens, num_q_heads, head_dim] in q's type, contiguous, and
 * lse fp32 [num_tokens, num_q_heads] (may be null) are written in full for
 * tokens below cu_q[num_seqs]; tokens behind it are left as they were.
 * Logits, softmax statistics and sums are fp32; the weights enter the second
 * product as 16-bit values (csa_cache_attend_rows.cu).
 *
 * Results are the same from call to call; the order of sums depends on the
 * sizes and lengths of the call alone. Workspace comes from the library's
 * stream-ordered pool. num_tokens == 0 launches nothing. num_tokens * num_q_heads
 * < 2^31.
 */
csa_status_t csa_cache_attend(const csa_cache_t* cache, const void* q, int32_t dtype,
                              int64_t num_tokens, int32_t num_q_heads, int64_t q_token_stride,
                              int64_t q_head_stride, int32_t kv_heads, int32_t shared,
                              float sm_scale, const int32_t* page_table, int32_t num_seqs,
                              int32_t max_pages, const int32_t* seq_lens, const int32_t* cu_q,
                              const int32_t* visible, void* out, float* lse,
                              cudaStream_t stream);

/*
 * Page handling. page_refs int32 [num_pages] counts the sequences that hold a
 * page (0: free). A sequence holds the pages of its table row, a run of
 * entries >= 0 from the row's start; every function keeps that form. New pages
 * are always the lowest-numbered free ones, in the order of the call's list
 * and then of the row, so results do not depend on timing.
 *
 * `status` is a caller-owned int32 device word that a call ORs bits into
 * (the caller zeroes it first and reads it when convenient). A call that
 * sets a bit other than CSA_CACHE_BAD_PAGE changes nothing else:
 */
#define CSA_CACHE_BAD_SEQ 1     /* a sequence index outside [0, num_seqs)           */
#define CSA_CACHE_DUPLICATE 2   /* an index twice, or one that is child and parent  */
#define CSA_CACHE_BUSY 4        /* a child that holds rows or pages                 */
#define CSA_CACHE_EXHAUSTED 8   /* fewer free pages than needed                     */
#define CSA_CACHE_TABLE_FULL 16 /* more rows than a table row has room for          */
#define CSA_CACHE_BAD_PAGE 32   /* a held page outside [0, num_pages): skipped      */

/*
 * Copies pages src[i] -> dst[i] (data and scales of all heads), i < n. The
 * destinations must be distinct and no destination may be a source of
 * another pair (their contents are unspecified otherwise). Pairs with a page
 * outside the pool, and src == dst, are skipped. One launch; n == 0 none.
 */
csa_status_t csa_cache_copy_pages(const csa_cache_t* cache, const int32_t* src,
                                  const int32_t* dst, int32_t n, cudaStream_t stream);

/*
 * Makes child i an equal of parent i: the same length and the same pages for
 * the rows it holds, whose counts grow by one; nothing is copied. Children
 * must be empty (length 0, no pages). A parent may have several children.
 */
csa_status_t csa_cache_fork(int32_t* page_table, int32_t* seq_lens, int32_t* page_refs,
                            int32_t num_seqs, int32_t max_pages, int32_t num_pages,
                            int32_t page_size, const int32_t* parents, const int32_t* children,
                            int32_t n, int32_t* status, cudaStream_t stream);

/*
 * Makes room for rows[i] more rows of sequence seqs[i]: allocates the pages
 * that are missing, and replaces pages that the new rows will be written to
 * and that other sequences hold too by a copy (copy on write). If all holders
 * of a page are in the list, the last of them in list order keeps it. Lengths
 * do not change. rows[i] <= 0 asks for nothing. All or nothing.
 */
csa_status_t csa_cache_reserve(const csa_cache_t* cache, int32_t* page_table,
                               const int32_t* seq_lens, int32_t* page_refs, int32_t num_seqs,
                               int32_t max_pages, const int32_t* seqs, const int32_t* rows,
                               int32_t n, int32_t* status, cudaStream_t stream);

/*
 * Ends sequences: their pages' counts fall by one, their table rows become -1
 * and their lengths 0. An index outside [0, num_seqs) is skipped; one that is
 * listed twice counts once.
 */
csa_status_t csa_cache_free(int32_t* page_table, int32_t* seq_lens, int32_t* page_refs,
                            int32_t num_seqs, int32_t max_pages, int32_t num_pages,
                            const int32_t* seqs, int32_t n, cudaStream_t stream);

/*
 * Moves the L held pages to the pool's front: the k-th held page at or above
 * L goes to the k-th free page below L; counts and tables follow. The pages
 * behind L are free afterwards (their contents stay). live (int32 device
 * word, may be null) gets L.
 */
csa_status_t csa_cache_compact(const csa_cache_t* cache, int32_t* page_table, int32_t* page_refs,
                               int32_t num_seqs, int32_t max_pages, int32_t* live,
                               cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA_CACHE_H */
