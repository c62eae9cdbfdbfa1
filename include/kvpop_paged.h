/*
 * kvpop_paged.h -- the fixed-budget KV cache in pages: filling it from a
 * prompt, appending tokens with eviction by accumulated attention weight, and
 * one decode step of attention over it (B200, sm_100a).
 *
 * kvpop.h holds the rules that apply here too: ownership, stream order, the
 * current device, errors, status words, kvpop_last_error, NVTX ranges.  The
 * calls are part of libkvpop.so.
 *
 * Where kvpop_compact_kv and kvpop_decode_attention keep one block
 * [batch, n_kv_heads, capacity, head_dim] per cache, a paged cache takes its
 * slots from a pool of pages shared by all sequences.  Slot c of row (b, h),
 * c < capacity, is
 *
 *   page = page_table[b * max_pages + c / page_size],  offset = c % page_size
 *   K    = k_pages + page * k_stride[0] + h * k_stride[1] + offset * k_stride[2]   (elements; head_dim contiguous)
 *   pos, weight at [page, h, offset] of contiguous [n_pages, n_kv_heads, page_size] arrays
 *
 * so pages laid out head by head or token by token, and K and V side by side
 * in one pool, are all described by strides.  The first count[b, h] slots of
 * a row are in use, in any order of positions; what lies behind them in a
 * page is neither read into a result nor written.
 *
 * 8-bit caches (KVPOP_PAGED_E4M3) hold K / k_scale[h] and V / v_scale[h],
 * divided in fp32, clipped to +-448 and rounded to nearest even; a NULL scale
 * is 1.  Scales must be finite and > 0.
 *
 * Page numbers are device data, so the kernels check them: an entry outside
 * [0, n_pages) that a call needs is never used as an address.  Its slots take
 * no part (attention), are left unwritten (compaction, append) and are not
 * evicted (append), and *dev_status, if given and still 0, receives
 * KVPOP_ERR_BOUNDS | site << 8 | kernel << 16 for kvpop_check_device_status.
 * Weights are the caller's data as much as the library's: between calls they
 * may be replaced, by a scorer's output say, and appends evict by whatever is
 * there.  An append sets the weight of each new token's slot to 0.
 * A page may not appear twice among the rows that one call writes (the weights
 * count as written by an attention that accumulates); rows that are only read
 * may share pages, such as those of a common prefix.  Positions stay below 2^31.
 */
#ifndef KVPOP_PAGED_H_
#define KVPOP_PAGED_H_

#include "kvpop.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KVPOP_PAGED_BF16 = 0,
  KVPOP_PAGED_E4M3 = 1
} kvpop_paged_dtype;

/* A paged cache.  Every pointer is device memory except the struct itself.
 * pos_pages, weight_pages, seen and the scales may be NULL where a call does
 * not need them. */
typedef struct {
  void* k_pages;              /* 16-byte aligned, as are all strides in bytes */
  void* v_pages;
  int64_t k_stride[3];        /* elements between pages, heads, slots; >= 0, pages and slots below 4 GiB */
  int64_t v_stride[3];
  int32_t* pos_pages;         /* [n_pages, n_kv_heads, page_size]: position of the token in a slot; 16-byte aligned */
  float* weight_pages;        /* the same layout: attention weight it has accumulated; 16-byte aligned */
  const float* k_scale;       /* [n_kv_heads] */
  const float* v_scale;
  const int32_t* page_table;  /* [batch, max_pages] */
  int32_t* count;             /* [batch, n_kv_heads]: slots in use; < 0 marks a row that takes no part */
  int32_t* seen;              /* [batch, n_kv_heads]: tokens the sequence has had, the next one's position */
  int32_t n_pages;
  int32_t page_size;          /* a power of two, 8 .. 1024 */
  int32_t max_pages;          /* entries of a page-table row */
  int32_t batch;              /* 1 .. 65535 */
  int32_t n_kv_heads;         /* 1 .. 1024 */
  int32_t head_dim;           /* 64 or 128 */
  int32_t capacity;           /* slots a row may use: 1 .. min(max_pages * page_size, 131072) */
  int32_t dtype;              /* kvpop_paged_dtype */
} kvpop_paged_cache;

/* Compaction into pages: per sequence b and KV head h, the positions with
 * keep = 1 fill slots 0, 1, ... in increasing order, up to capacity; the
 * rest are dropped.  pos, count (slots used) and seen (the sequence's length)
 * are written, and weight = score (the attention a token has received so far:
 * kvpop_future_target with window 0 gives exactly that for a prompt) or 0.
 *   k, v         bf16 [T, n_kv_heads, head_dim], 16-byte aligned (NULL with T = 0)
 *   keep         uint8 [n_kv_heads, T], or NULL to keep every position
 *   score        fp32 [n_kv_heads, T], or NULL for 0 (needs cache->weight_pages otherwise)
 *   cu_seqlens   HOST int32 [batch + 1]; batch = cache->batch at most 512, sequences of at most 131072
 *                tokens; cu_seqlens[batch] = total_tokens
 * cache->pos_pages, weight_pages and seen are written where they are given. */
KVPOP_API kvpop_status kvpop_paged_compact_kv(const void* k, const void* v, const uint8_t* keep, const float* score,
                                              const int32_t* cu_seqlens, int32_t total_tokens,
                                              const kvpop_paged_cache* cache, int32_t* dev_status, void* stream);

/* Appends m_b new tokens to every sequence b, evicting when a row is full.
 * With n = min(count, capacity) slots in use, the first capacity - n of them
 * go to slots n, n + 1, ...; each further one replaces the slot of the token
 * that ranks last by accumulated weight, in the order of kvpop_keep_mask
 * (NaN below every number, -0 equal to +0, of equal weights the larger
 * position goes first).  Tokens at positions < sinks and those that are among
 * the `window` most recent once the new ones are in (position >= seen + m_b -
 * window) are never replaced.  The replaced slots, in increasing order, take
 * the remaining new tokens in theirs.  A new token's position is seen + its
 * place among the m_b, its weight 0.  count and seen are advanced.
 *   k_new, v_new   bf16 [T_new, n_kv_heads, head_dim], token_stride elements between tokens
 *                  (a multiple of 8, below 4 GiB; head_dim and heads contiguous), 16-byte aligned
 *   cu_new         HOST int32 [batch + 1], offsets of each sequence's new tokens (batch at most 512 then);
 *                  NULL = one token each
 *   window, sinks  every m_b <= max(window, 1); capacity >= sinks + max(window, 1)
 *   evicted        int32 [T_new, n_kv_heads] or NULL: the position that a token displaced, -1 where it took a
 *                  free slot, -2 where it was not stored
 * Rows with count < 0 are left as they are.  A token without a slot (which
 * needs a bad page, or positions that break the rules above) is not stored
 * and reported in *dev_status.  The choice is exact and depends on no order of
 * execution.  Nothing but counts, positions and weights on the device decides,
 * so the call can be captured in a graph and replayed. */
KVPOP_API kvpop_status kvpop_paged_append_kv(const void* k_new, const void* v_new, int64_t token_stride,
                                             const int32_t* cu_new, const kvpop_paged_cache* cache, int32_t window,
                                             int32_t sinks, int32_t* evicted, int32_t* dev_status, void* stream);

/* Device workspace (bytes) of kvpop_paged_decode_attention; 0 for a cache
 * that the call would refuse. */
KVPOP_API size_t kvpop_paged_decode_workspace_bytes(const kvpop_paged_cache* cache, int32_t n_q_heads,
                                                    int32_t accumulate);

/* One decode step over the paged cache: for sequence b, query head g and its
 * KV head h = g / G (G = n_q_heads / n_kv_heads, at most 1,024),
 *   s[c]      = scale * q[b, g, :] . K[c, :],  c < n = clamp(count[b, h], 0, capacity)
 *   lse[b, g] = ln sum_c exp(s[c]),  out[b, g, :] = sum_c exp(s[c] - lse) V[c, :]
 * and, with accumulate != 0, weight[c] += sum over the group's heads of
 * exp(s[c] - lse).  n = 0 gives out = 0 and lse = -inf.
 *   q          bf16 [batch, n_q_heads, head_dim], q_stride elements between sequences (a multiple
 *              of 8), 16-byte aligned
 *   out        bf16 [batch, n_q_heads, head_dim], 16-byte aligned
 *   lse        fp32 [batch, n_q_heads] or NULL
 *   workspace  >= kvpop_paged_decode_workspace_bytes bytes, 256-byte aligned; contents on entry are
 *              ignored; calls that overlap on the GPU need one each
 * Scores, softmax statistics and sums are fp32; a probability enters the
 * second product as a high and a low 16-bit part (16 bits of it and more), so
 * out is rounded once, to bf16. */
KVPOP_API kvpop_status kvpop_paged_decode_attention(const void* q, int64_t q_stride, int32_t n_q_heads,
                                                    const kvpop_paged_cache* cache, float scale, int32_t accumulate,
                                                    void* out, float* lse, void* workspace, size_t workspace_bytes,
                                                    int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVPOP_PAGED_H_ */
