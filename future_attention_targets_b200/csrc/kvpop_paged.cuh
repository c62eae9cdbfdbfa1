// Parameter blocks and device helpers of the paged-cache kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kvpop_debug.cuh"
#include "kvpop_host.h"
#include "kvpop_sched.h"

namespace kvpop {

// Kernel numbers in status words, after those of kvpop_debug.cuh.
constexpr int32_t DBG_PAGED_DECODE = 11;
constexpr int32_t DBG_PAGED_JOIN = 12;
constexpr int32_t DBG_PAGED_APPEND = 13;
constexpr int32_t DBG_PAGED_COMPACT = 14;

// The cache as the kernels see it: byte pointers and byte strides.
struct PagedView {
  uint8_t* k;
  uint8_t* v;
  int64_t k_page, k_head, k_slot;   // bytes
  int64_t v_page, v_head, v_slot;
  int32_t* pos;
  float* weight;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int32_t* count;
  int32_t* seen;
  int32_t n_pages, page_shift, max_pages, batch, n_kv_heads, capacity;
};

struct PagedDecodeParams {
  PagedView c;
  const uint16_t* q;
  int64_t q_stride;       // elements between sequences
  uint16_t* out;          // bf16 [B, H_q, d]
  float* lse;             // [B, H_q] or null
  int2* item_parts;       // [items]: the first CTA that holds slots of an item, and how many do
  float* part_o;          // [CTAs, 2, 16, d]: parts of the items that a CTA's share goes on with (0) and starts (1)
  float2* part_ml;        // [CTAs, 2, 16]: their maxima (log2 units) and sums
  float* row_lse2;        // [B * H_q]: lse in log2 units of items that one CTA did
  float* scores;          // [B * H_q, score_pitch], log2 units; null = weights not accumulated
  int32_t* status;
  int32_t* dbg;
  int32_t n_q_heads, group, head_chunks, ctas, whole, score_pitch;   // whole: a CTA per item, and no second kernel
  float scale_log2;
};

// How a decode step's items are dealt out.
struct DecodeSplit {
  int ctas;
  bool whole;
};

struct PagedAppendParams {
  PagedView c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t token_stride;   // elements
  int32_t* evicted;
  int32_t* status;
  int32_t* dbg;
  int32_t window, sinks, one_each, slice;   // slice: slots of a row that one CTA of its cluster looks at
  int32_t start[kMaxSeqs + 1];
};

struct PagedCompactParams {
  PagedView c;
  const uint16_t* k;
  const uint16_t* v;
  const uint8_t* keep;    // or null
  const float* score;     // or null
  int32_t* status;
  int32_t* dbg;
  int32_t total_tokens, block;   // block: positions of one CTA
  int32_t start[kMaxSeqs + 1];
};

// The kernels are programmatic dependents: they may be resident while the one before still writes what they read.  The
// wait orders ordinary loads behind those writes, not non-coherent ones (__ldg), so there are none of those.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Page of entry e of sequence b's table row, or -1 (and a report) where the
// table has no page of the pool there.
__device__ __forceinline__ int32_t page_of(const PagedView& c, int32_t b, int32_t e, int32_t* status, int32_t kernel,
                                           int32_t site) {
  if (e < 0 || e >= c.max_pages) return -1;
  const int32_t page = c.table[static_cast<int64_t>(b) * c.max_pages + e];
  if (static_cast<uint32_t>(page) < static_cast<uint32_t>(c.n_pages)) return page;
  debug_fail(status, kernel, site);
  return -1;
}

// Rows to write, in shared memory: token `tok` of the sources (from the first one of the list on) goes to offset
// `off` of `page`; a page < 0 is skipped.
struct RowEntry {
  int32_t page;
  uint32_t off_tok;       // off | tok << 10: pages have at most 1,024 slots
};
__device__ __forceinline__ RowEntry row_entry(int page, int off, int tok) {
  return {page, static_cast<uint32_t>(off) | (static_cast<uint32_t>(tok) << 10)};
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) { return (static_cast<uint64_t>(hi) << 32) | lo; }
__device__ __forceinline__ uint64_t twice(float x) { return pair_of(__float_as_uint(x), __float_as_uint(x)); }
// Two fp32 values to two e4m3, nearest even, clipped to +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(uint64_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(r)
      : "f"(__uint_as_float(static_cast<uint32_t>(x >> 32))), "f"(__uint_as_float(static_cast<uint32_t>(x))));
  return r;
}

// What the rows of an 8-bit cache are divided by, and the division: the correctly rounded fp32 quotient, two at a
// time.  x is clipped to just past +-464 scale, beyond which everything rounds to +-448, so that nothing overflows;
// the product of -x with the negated rounded reciprocal is then corrected by its exact remainder (P. Markstein, IBM
// J. Res. Dev. 34(1), 1990), with signs that keep -0.  That is correctly rounded wherever the remainder does not
// underflow, which for scales of 2^-60 to 2^60 is every quotient that e4m3 does not flush to 0.  Other scales divide.
// With a division for every element an 8-bit cache's compaction was bound by it (8 prompts, 100,003 tokens: 127 us),
// with two conversions to enclose the quotient by those (104 us).
struct Divisor {
  float scale;
  bool divide;
  uint32_t clip, clip_neg;       // bf16x2
  uint64_t neg_inv, scale2;
};
__device__ __forceinline__ Divisor divisor_of(float scale) {
  Divisor d;
  d.scale = scale;
  d.divide = !(scale >= 0x1p-60f && scale <= 0x1p60f);
  d.clip = (__float_as_uint(500.f * scale) >> 16) * 0x10001u;      // bf16, rounded down: at least 496 scale
  d.clip_neg = d.clip | 0x80008000u;
  d.neg_inv = twice(-__frcp_rn(scale));
  d.scale2 = twice(scale);
  return d;
}
__device__ __forceinline__ uint2 to_e4m3x8(const uint4& in, const Divisor& by) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t r[4];
  if (by.divide) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      r[e] = e4m3x2(pair_of(__float_as_uint(__fdiv_rn(__uint_as_float(w[e] << 16), by.scale)),
                            __float_as_uint(__fdiv_rn(__uint_as_float(w[e] & 0xffff0000u), by.scale))));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t y = w[e] ^ 0x80008000u;
      asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(by.clip));
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(by.clip_neg));
      const uint64_t neg_x = pair_of(y << 16, y & 0xffff0000u);
      const uint64_t q = mul2(neg_x, by.neg_inv);
      r[e] = e4m3x2(fma2(fma2(q, by.scale2, neg_x), by.neg_inv, q));
    }
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Copies the K and V rows of `n` list entries of head h, bf16 to bf16 or to e4m3.  A warp takes an entry (two with 64
// dims) at a time, its lanes the 16-byte words of K's row, then V's, with kUnroll entries in flight.
template <int D, bool kF8, int kThreads, int kUnroll>
__device__ __forceinline__ void copy_rows(const PagedView& c, const uint16_t* k, const uint16_t* v,
                                          int64_t token_stride, int h, const RowEntry* list, int n) {
  constexpr int kWords = D / 8;             // 16-byte words of a bf16 row
  constexpr int kPer = 32 / (2 * kWords);   // entries of a warp at a time
  constexpr int kStep = kThreads / 32 * kPer;
  const int lane = threadIdx.x & 31;
  const int w = lane % kWords;
  const bool is_v = (lane / kWords) & 1;
  const uint8_t* src = reinterpret_cast<const uint8_t*>((is_v ? v : k) + static_cast<int64_t>(h) * D + 8 * w);
  uint8_t* dst = (is_v ? c.v + h * c.v_head : c.k + h * c.k_head) + (kF8 ? 8 : 16) * w;
  // The host keeps these within 32 bits, so that an address is one or two wide multiply-adds.
  const uint32_t token_bytes = static_cast<uint32_t>(token_stride) * 2u;
  const uint32_t page_bytes = static_cast<uint32_t>(is_v ? c.v_page : c.k_page);
  const uint32_t slot_bytes = static_cast<uint32_t>(is_v ? c.v_slot : c.k_slot);
  Divisor by = {};
  if constexpr (kF8) {
    const float* s = is_v ? c.v_scale : c.k_scale;
    by = divisor_of(s != nullptr ? s[h] : 1.f);
  }
  for (int base = threadIdx.x / 32 * kPer + lane / (2 * kWords); base < n; base += kStep * kUnroll) {
    uint4 buf[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kStep;
      if (i < n)
        buf[u] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<uint64_t>(list[i].off_tok >> 10) * token_bytes));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * kStep;
      if (i < n) {
        const RowEntry e = list[i];
        if (e.page >= 0) {
          uint8_t* to = dst + static_cast<uint64_t>(static_cast<uint32_t>(e.page)) * page_bytes +
                        static_cast<uint64_t>(e.off_tok & 1023u) * slot_bytes;
          if constexpr (kF8) *reinterpret_cast<uint2*>(to) = to_e4m3x8(buf[u], by);
          else *reinterpret_cast<uint4*>(to) = buf[u];
        }
      }
    }
  }
}

// The contexts in which a kernel's limit of dynamic shared memory has been raised, by id: a context loads the kernel
// anew, without the limit.  Ids that share a place raise it again each time they take turns.
struct SmemReady {
  std::atomic<unsigned long long> context[16];
};

// Raises the limit in the current context, once.  Another thread may do it again at the same time: that changes nothing.
template <class Kern>
static cudaError_t allow_smem(Kern kern, size_t bytes, SmemReady& ready) {
  const unsigned long long id = current_context_id();
  if (id != 0 && ready.context[id % 16].load(std::memory_order_relaxed) == id) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && id != 0) ready.context[id % 16].store(id, std::memory_order_relaxed);
  return e;
}

// Launch as a programmatic dependent of the stream's previous kernel, with
// clusters of `cluster` CTAs along x when that is more than one.
template <class Kern, class Params>
static cudaError_t launch_paged(Kern kern, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream,
                                const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace kvpop
