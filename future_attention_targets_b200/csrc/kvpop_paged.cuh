// Parameter blocks and device helpers of the paged-cache kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kvpop_debug.cuh"
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
  float* part_o;          // [B * H_q, n_split, d]
  float2* part_ml;        // [B * H_q, n_split]: running max (log2 units), sum
  float* scores;          // [B * H_q, score_pitch], log2 units; null = weights not accumulated
  int32_t* status;
  int32_t* dbg;
  int32_t n_q_heads, group, head_chunks, split_slots, n_split, score_pitch;
  float scale_log2;
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

// A batch of rows to write: token l_tok[i] of the sources goes to slot l_off[i]
// of page l_page[i]; l_page[i] < 0 is skipped.
struct RowList {
  int32_t* page;
  int32_t* off;
  int32_t* tok;
};

// Copies the K and V rows of `n` list entries of head h, bf16 to bf16 or to
// e4m3, 16 bytes of input per thread and step, kUnroll steps in flight.
template <int D, bool kF8, int kThreads, int kUnroll>
__device__ __forceinline__ void copy_rows(const PagedView& c, const uint16_t* k, const uint16_t* v,
                                          int64_t token_stride, int h, const RowList& list, int n) {
  constexpr int kWords = D / 8;             // 16-byte words of a bf16 row
  float ks = 1.f, vs = 1.f;
  if constexpr (kF8) {
    if (c.k_scale != nullptr) ks = c.k_scale[h];
    if (c.v_scale != nullptr) vs = c.v_scale[h];
  }
  const int total = n * 2 * kWords;
  for (int base = threadIdx.x; base < total; base += kThreads * kUnroll) {
    uint4 buf[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int idx = base + u * kThreads;
      const int i = idx / (2 * kWords), w = idx % kWords;
      if (idx < total && list.page[i] >= 0) {
        const uint16_t* src = (idx / kWords) & 1 ? v : k;
        buf[u] = __ldg(reinterpret_cast<const uint4*>(src + list.tok[i] * token_stride + static_cast<int64_t>(h) * D + 8 * w));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int idx = base + u * kThreads;
      const int i = idx / (2 * kWords), w = idx % kWords;
      if (idx < total && list.page[i] >= 0) {
        const bool is_v = (idx / kWords) & 1;
        uint8_t* dst = is_v ? c.v + list.page[i] * c.v_page + h * c.v_head + list.off[i] * c.v_slot
                            : c.k + list.page[i] * c.k_page + h * c.k_head + list.off[i] * c.k_slot;
        if constexpr (kF8) {
          const float scale = is_v ? vs : ks;
          const uint32_t in[4] = {buf[u].x, buf[u].y, buf[u].z, buf[u].w};
          uint32_t out[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = make_float2(__fdiv_rn(__uint_as_float(in[e] << 16), scale),
                                         __fdiv_rn(__uint_as_float(in[e] & 0xffff0000u), scale));
            // Rounds to nearest even and saturates to +-448; NaN stays NaN.
            out[e / 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) << (16 * (e & 1));
          }
          *reinterpret_cast<uint2*>(dst + 8 * w) = make_uint2(out[0], out[1]);
        } else {
          *reinterpret_cast<uint4*>(dst + 16 * w) = buf[u];
        }
      }
    }
  }
}

// Raises a kernel's dynamic shared memory limit on the current device, once per device (`done`: one bit each).
// Another thread may do it again at the same time: that changes nothing.
template <class Kern>
static cudaError_t allow_smem(Kern kern, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
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
