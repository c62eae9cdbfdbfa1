// Host side of the paged cache's C ABI (include/kvpop_paged.h): argument
// validation, byte strides, workspace layout and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <nvtx3/nvToolsExt.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "kvpop_host.h"
#include "kvpop_paged.cuh"
#include "kvpop_paged.h"

namespace kvpop {
cudaError_t launch_paged_decode(const PagedDecodeParams& p, int head_dim, bool f8, cudaStream_t stream);
cudaError_t launch_paged_append(PagedAppendParams& p, int head_dim, bool f8, cudaStream_t stream);
cudaError_t launch_paged_compact(PagedCompactParams& p, int head_dim, bool f8, cudaStream_t stream);
DecodeSplit paged_split(int64_t items, int capacity, int head_dim, bool f8, bool wide, bool may_be_whole);
}  // namespace kvpop

using namespace kvpop;

namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

constexpr int kMaxCapacity = 131072;
constexpr int kMaxBatch = 65535;
constexpr int kMaxKvHeads = 1024;
constexpr int kMaxQHeads = 1 << 16;
constexpr int kMaxGroup = 1024;       // query heads per KV head

kvpop_status fail(kvpop_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return host_fail(st, buf);
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

kvpop_status check_cache(const kvpop_paged_cache* c) {
  if (c == nullptr) return fail(KVPOP_ERR_INVALID_ARG, "cache is NULL");
  if (c->dtype != KVPOP_PAGED_BF16 && c->dtype != KVPOP_PAGED_E4M3)
    return fail(KVPOP_ERR_INVALID_ARG, "cache dtype %d is neither bf16 nor e4m3", c->dtype);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(KVPOP_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", c->head_dim);
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(KVPOP_ERR_UNSUPPORTED, "page_size %d not supported (a power of two, 8 .. 1024)", c->page_size);
  if (c->batch < 1 || c->n_kv_heads < 1 || c->n_pages < 1 || c->max_pages < 1)
    return fail(KVPOP_ERR_INVALID_ARG, "batch, n_kv_heads, n_pages and max_pages must be >= 1");
  if (c->batch > kMaxBatch || c->n_kv_heads > kMaxKvHeads)
    return fail(KVPOP_ERR_UNSUPPORTED, "at most %d sequences and %d KV heads", kMaxBatch, kMaxKvHeads);
  if (c->capacity < 1 || c->capacity > static_cast<int64_t>(c->max_pages) * c->page_size)
    return fail(KVPOP_ERR_INVALID_ARG, "capacity %d is not within 1 .. max_pages * page_size", c->capacity);
  if (c->capacity > kMaxCapacity)
    return fail(KVPOP_ERR_UNSUPPORTED, "capacity %d exceeds %d slots", c->capacity, kMaxCapacity);
  if (c->k_pages == nullptr || c->v_pages == nullptr || c->page_table == nullptr || c->count == nullptr)
    return fail(KVPOP_ERR_INVALID_ARG, "k_pages, v_pages, page_table or count is NULL");
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->pos_pages, 16) || !aligned(c->weight_pages, 16))
    return fail(KVPOP_ERR_INVALID_ARG, "the pages must be 16-byte aligned");
  const int elt = c->dtype == KVPOP_PAGED_E4M3 ? 1 : 2;
  for (int i = 0; i < 3; ++i) {
    const int64_t s[2] = {c->k_stride[i], c->v_stride[i]};
    for (int64_t x : s) {
      if (x < 0 || x > (int64_t(1) << 56) || x * elt % 16 != 0)
        return fail(KVPOP_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes");
      if (i != 1 && x * elt >= (int64_t(1) << 32))
        return fail(KVPOP_ERR_UNSUPPORTED, "strides between pages and between slots must be below 4 GiB");
    }
  }
  return KVPOP_OK;
}

PagedView view_of(const kvpop_paged_cache& c) {
  const int64_t elt = c.dtype == KVPOP_PAGED_E4M3 ? 1 : 2;
  PagedView v = {};
  v.k = static_cast<uint8_t*>(c.k_pages);
  v.v = static_cast<uint8_t*>(c.v_pages);
  v.k_page = c.k_stride[0] * elt, v.k_head = c.k_stride[1] * elt, v.k_slot = c.k_stride[2] * elt;
  v.v_page = c.v_stride[0] * elt, v.v_head = c.v_stride[1] * elt, v.v_slot = c.v_stride[2] * elt;
  v.pos = c.pos_pages;
  v.weight = c.weight_pages;
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.table = c.page_table;
  v.count = c.count;
  v.seen = c.seen;
  v.n_pages = c.n_pages;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  v.max_pages = c.max_pages;
  v.batch = c.batch;
  v.n_kv_heads = c.n_kv_heads;
  v.capacity = c.capacity;
  return v;
}

// Offsets of `batch` runs in a packed array: 0 first, never decreasing.
kvpop_status check_offsets(const int32_t* cu, int batch, const char* name) {
  if (batch > kMaxSeqs)
    return fail(KVPOP_ERR_UNSUPPORTED, "%s: %d sequences exceed the %d-sequence limit", name, batch, kMaxSeqs);
  if (cu[0] != 0) return fail(KVPOP_ERR_INVALID_ARG, "%s[0] must be 0 (got %d)", name, cu[0]);
  for (int b = 0; b < batch; ++b)
    if (cu[b + 1] < cu[b]) return fail(KVPOP_ERR_INVALID_ARG, "%s decreases at %d", name, b);
  return KVPOP_OK;
}

// How a decode step is cut up, and where its parts lie in the workspace.
struct DecodePlan {
  int head_chunks, score_pitch;
  DecodeSplit split;
  size_t first, ml, o, lse2, scores, bytes;
};

DecodePlan plan_decode(const kvpop_paged_cache& c, int n_q_heads, bool accumulate) {
  DecodePlan d = {};
  const int group = n_q_heads / c.n_kv_heads;
  d.head_chunks = (group + 15) / 16;
  const int64_t items = static_cast<int64_t>(c.batch) * c.n_kv_heads * d.head_chunks;
  // Heads of several chunks add to the same weights: the second kernel sums those in a fixed order.
  d.split = paged_split(items, c.capacity, c.head_dim, c.dtype == KVPOP_PAGED_E4M3, group > 8,
                        d.head_chunks == 1 || !accumulate);
  d.score_pitch = (c.capacity + 63) / 64 * 64;
  const size_t heads = static_cast<size_t>(c.batch) * n_q_heads;
  if (!d.split.whole) {
    d.first = round256(items * sizeof(int2));
    d.ml = round256(static_cast<size_t>(d.split.ctas) * 2 * 16 * sizeof(float2));
    d.o = round256(static_cast<size_t>(d.split.ctas) * 2 * 16 * c.head_dim * sizeof(float));
    d.lse2 = accumulate ? round256(heads * sizeof(float)) : 0;
  }
  d.scores = accumulate ? round256(heads * d.score_pitch * sizeof(float)) : 0;
  d.bytes = d.first + d.ml + d.o + d.lse2 + d.scores;
  return d;
}

kvpop_status check_q_heads(const kvpop_paged_cache& c, int32_t n_q_heads) {
  if (n_q_heads < 1 || n_q_heads % c.n_kv_heads != 0)
    return fail(KVPOP_ERR_INVALID_ARG, "n_q_heads (%d) is not a multiple of n_kv_heads (%d)", n_q_heads, c.n_kv_heads);
  if (n_q_heads > kMaxQHeads) return fail(KVPOP_ERR_UNSUPPORTED, "at most %d query heads", kMaxQHeads);
  if (n_q_heads / c.n_kv_heads > kMaxGroup)
    return fail(KVPOP_ERR_UNSUPPORTED, "at most %d query heads per KV head", kMaxGroup);
  if (static_cast<int64_t>(c.batch) * n_q_heads >= (int64_t(1) << 27))
    return fail(KVPOP_ERR_UNSUPPORTED, "too many (sequence, head) items for one launch");
  if (plan_decode(c, n_q_heads, true).split.ctas == 0 || plan_decode(c, n_q_heads, false).split.ctas == 0)
    return fail(KVPOP_ERR_UNSUPPORTED, "too many slots for one launch");
  return KVPOP_OK;
}

}  // namespace

extern "C" {

kvpop_status kvpop_paged_compact_kv(const void* k, const void* v, const uint8_t* keep, const float* score,
                                    const int32_t* cu_seqlens, int32_t total_tokens, const kvpop_paged_cache* cache,
                                    int32_t* dev_status, void* stream) {
  Range range(__func__);
  kvpop_status st;
  if ((k == nullptr || v == nullptr) && total_tokens != 0) return fail(KVPOP_ERR_INVALID_ARG, "k or v is NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(KVPOP_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (cu_seqlens == nullptr) return fail(KVPOP_ERR_INVALID_ARG, "cu_seqlens is NULL");
  if ((st = check_cache(cache)) != KVPOP_OK) return st;
  if (score != nullptr && cache->weight_pages == nullptr)
    return fail(KVPOP_ERR_INVALID_ARG, "score is given but the cache has no weight_pages");
  if ((st = check_offsets(cu_seqlens, cache->batch, "cu_seqlens")) != KVPOP_OK) return st;
  if (cu_seqlens[cache->batch] != total_tokens)
    return fail(KVPOP_ERR_INVALID_ARG, "cu_seqlens[batch] (%d) != total_tokens (%d)", cu_seqlens[cache->batch],
                total_tokens);
  for (int b = 0; b < cache->batch; ++b)
    if (cu_seqlens[b + 1] - cu_seqlens[b] > kMaxCapacity)
      return fail(KVPOP_ERR_UNSUPPORTED, "sequence %d has %d tokens (limit %d)", b, cu_seqlens[b + 1] - cu_seqlens[b],
                  kMaxCapacity);
  if ((st = host_device()) != KVPOP_OK) return st;
  PagedCompactParams p = {};
  p.c = view_of(*cache);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.keep = keep;
  p.score = score;
  p.status = dev_status;
  p.dbg = host_debug_word();
  p.total_tokens = total_tokens;
  std::copy(cu_seqlens, cu_seqlens + cache->batch + 1, p.start);
  const cudaError_t e = launch_paged_compact(p, cache->head_dim, cache->dtype == KVPOP_PAGED_E4M3,
                                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVPOP_OK : host_cuda_fail(e, "paged compaction launch");
}

kvpop_status kvpop_paged_append_kv(const void* k_new, const void* v_new, int64_t token_stride, const int32_t* cu_new,
                                   const kvpop_paged_cache* cache, int32_t window, int32_t sinks, int32_t* evicted,
                                   int32_t* dev_status, void* stream) {
  Range range(__func__);
  kvpop_status st;
  if (k_new == nullptr || v_new == nullptr) return fail(KVPOP_ERR_INVALID_ARG, "k_new or v_new is NULL");
  if (!aligned(k_new, 16) || !aligned(v_new, 16))
    return fail(KVPOP_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
  if ((st = check_cache(cache)) != KVPOP_OK) return st;
  if (token_stride < 0 || token_stride % 8 != 0)
    return fail(KVPOP_ERR_INVALID_ARG, "token_stride must be a non-negative multiple of 8 elements");
  if (token_stride >= (int64_t(1) << 31)) return fail(KVPOP_ERR_UNSUPPORTED, "token_stride must be below 4 GiB");
  if (cache->pos_pages == nullptr || cache->weight_pages == nullptr || cache->seen == nullptr)
    return fail(KVPOP_ERR_INVALID_ARG, "appending needs pos_pages, weight_pages and seen");
  if (window < 0 || sinks < 0) return fail(KVPOP_ERR_INVALID_ARG, "window and sinks must be >= 0");
  const int64_t most = std::max(window, 1);
  if (cache->capacity < sinks + most)
    return fail(KVPOP_ERR_INVALID_ARG, "capacity %d is less than sinks + max(window, 1)", cache->capacity);
  if (static_cast<int64_t>(cache->batch) * cache->n_kv_heads * 8 >= (int64_t(1) << 31))
    return fail(KVPOP_ERR_UNSUPPORTED, "too many rows for one launch");
  if (cu_new != nullptr) {
    if ((st = check_offsets(cu_new, cache->batch, "cu_new")) != KVPOP_OK) return st;
    for (int b = 0; b < cache->batch; ++b)
      if (cu_new[b + 1] - cu_new[b] > most)
        return fail(KVPOP_ERR_INVALID_ARG, "sequence %d appends %d tokens, more than max(window, 1)", b,
                    cu_new[b + 1] - cu_new[b]);
    if (cu_new[cache->batch] == 0) return KVPOP_OK;
  }
  if ((st = host_device()) != KVPOP_OK) return st;
  PagedAppendParams p = {};
  p.c = view_of(*cache);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.token_stride = token_stride;
  p.evicted = evicted;
  p.status = dev_status;
  p.dbg = host_debug_word();
  p.window = window;
  p.sinks = sinks;
  p.one_each = cu_new == nullptr;
  if (cu_new != nullptr) std::copy(cu_new, cu_new + cache->batch + 1, p.start);
  const cudaError_t e = launch_paged_append(p, cache->head_dim, cache->dtype == KVPOP_PAGED_E4M3,
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVPOP_OK : host_cuda_fail(e, "paged append launch");
}

size_t kvpop_paged_decode_workspace_bytes(const kvpop_paged_cache* cache, int32_t n_q_heads, int32_t accumulate) {
  if (check_cache(cache) != KVPOP_OK || check_q_heads(*cache, n_q_heads) != KVPOP_OK) return 0;
  return plan_decode(*cache, n_q_heads, accumulate != 0).bytes;
}

kvpop_status kvpop_paged_decode_attention(const void* q, int64_t q_stride, int32_t n_q_heads,
                                          const kvpop_paged_cache* cache, float scale, int32_t accumulate, void* out,
                                          float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                          void* stream) {
  Range range(__func__);
  kvpop_status st;
  if (q == nullptr || out == nullptr) return fail(KVPOP_ERR_INVALID_ARG, "q or out is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVPOP_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (!isfinite(scale) || !(scale > 0.f)) return fail(KVPOP_ERR_INVALID_ARG, "scale must be finite and > 0");
  if ((st = check_cache(cache)) != KVPOP_OK) return st;
  if ((st = check_q_heads(*cache, n_q_heads)) != KVPOP_OK) return st;
  if (q_stride < 0 || q_stride > (int64_t(1) << 40) || q_stride % 8 != 0)
    return fail(KVPOP_ERR_INVALID_ARG, "q_stride must be a non-negative multiple of 8 elements");
  if (accumulate != 0 && cache->weight_pages == nullptr)
    return fail(KVPOP_ERR_INVALID_ARG, "accumulating needs weight_pages");
  const DecodePlan d = plan_decode(*cache, n_q_heads, accumulate != 0);
  if (d.bytes > 0 && (workspace == nullptr || workspace_bytes < d.bytes))
    return fail(KVPOP_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu required",
                workspace == nullptr ? size_t(0) : workspace_bytes, d.bytes);
  if (!aligned(workspace, 256)) return fail(KVPOP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((st = host_device()) != KVPOP_OK) return st;
  PagedDecodeParams p = {};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.c = view_of(*cache);
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.item_parts = reinterpret_cast<int2*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + d.first);
  p.part_o = reinterpret_cast<float*>(ws + d.first + d.ml);
  p.row_lse2 = reinterpret_cast<float*>(ws + d.first + d.ml + d.o);
  p.scores = accumulate != 0 ? reinterpret_cast<float*>(ws + d.first + d.ml + d.o + d.lse2) : nullptr;
  p.status = dev_status;
  p.dbg = host_debug_word();
  p.n_q_heads = n_q_heads;
  p.group = n_q_heads / cache->n_kv_heads;
  p.head_chunks = d.head_chunks;
  p.ctas = d.split.ctas;
  p.whole = d.split.whole;
  p.score_pitch = d.score_pitch;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const cudaError_t e = launch_paged_decode(p, cache->head_dim, cache->dtype == KVPOP_PAGED_E4M3,
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVPOP_OK : host_cuda_fail(e, "paged decode attention launch");
}

}  // extern "C"
