// Appending tokens to the paged cache, with eviction of the tokens of least
// accumulated attention weight, sm_100a.
//
// A row (sequence, KV head) is handled by a cluster of 1 to 8 CTAs, each of
// which looks at a slice of the row's slots.  What a slot is worth is one
// 64-bit key, smaller = evicted earlier: the order-preserving bits of the
// weight (NaN lowest), then 2^31 - 1 - position; slots that may not go (sinks,
// recent tokens) have the key 2^64 - 1.  One token in, one out (the steady
// state of decoding) is an argmin over the keys.  Several out is an exact
// radix select of the e-th smallest key, digit by digit, over keys in shared
// memory: the cluster adds its histograms through distributed shared memory,
// and stops as soon as a digit's bucket is taken whole.  Everything is
// integer, so the result is exact and does not depend on any order.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvpop_paged.cuh"

namespace kvpop {

namespace cg = cooperative_groups;

constexpr int kPaThreads = 256;
constexpr int kPaWarps = kPaThreads / 32;
constexpr int kPaMaxSlice = 16384;     // keys one CTA holds at most (128 KiB); 8 x 16384 = the largest capacity
constexpr uint64_t kStays = ~0ull;

// Larger float -> larger key; -0 equals +0; NaN -> 0, below every number.
__device__ __forceinline__ uint32_t weight_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int D, bool kF8, bool kChunk>
__global__ void __launch_bounds__(kPaThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  extern __shared__ uint64_t keys[];                     // kChunk: this CTA's slice
  __shared__ uint64_t best_key[kPaWarps + 1];            // one out: minimum of each warp; [kPaWarps] = of the CTA
  __shared__ int32_t best_slot[kPaWarps + 1];
  __shared__ uint32_t hist[2][256];                      // kChunk: a pass's histogram, read by the cluster
  __shared__ uint32_t sel[3];
  __shared__ uint32_t taken_here;                        // kChunk: victims in this slice, read by the cluster
  __shared__ uint32_t warp_sum[kPaWarps];
  __shared__ int32_t l_page[kPaThreads], l_off[kPaThreads], l_tok[kPaThreads];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / ctas, b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int page_mask = (1 << p.c.page_shift) - 1;
  const int tok0 = p.one_each ? b : p.start[b];
  const int m = p.one_each ? 1 : p.start[b + 1] - tok0;
  if (m == 0) return;                                    // as for every branch on b or count: the whole cluster
  grid_wait();
  grid_launch_next();
  const int count = p.c.count[row], seen = p.c.seen[row];
  if (count < 0) {
    if (p.evicted != nullptr && cta == 0)
      for (int i = tid; i < m; i += kPaThreads) p.evicted[static_cast<int64_t>(tok0 + i) * p.c.n_kv_heads + h] = -2;
    return;
  }
  const int cap = p.c.capacity, n = min(count, cap), f = min(m, cap - n), e = m - f;
  // Position below which a token has left the recent window once the new ones are in.
  const int64_t recent = static_cast<int64_t>(seen) + m - p.window;
  const int s0 = min(n, cta * p.slice), s1 = min(n, s0 + p.slice);

  auto meta_at = [&](int page, int off) {
    return ((static_cast<int64_t>(page) * p.c.n_kv_heads + h) << p.c.page_shift) + off;
  };
  auto key_of = [&](float w, int pos) {
    const bool goes = pos >= p.sinks && pos < recent;
    return goes ? (static_cast<uint64_t>(weight_key(w)) << 32) | static_cast<uint32_t>(0x7fffffff - pos) : kStays;
  };
  // Calls use(slot, key) for the slots of this CTA's slice, 4 per thread and step (a page has at least 8 slots
  // and slices are multiples of 8, so four slots share a page and an aligned 16 bytes).
  auto for_keys = [&](auto&& use) {
    constexpr int kU = 4;
    for (int base = s0 + 4 * tid; base < s1; base += 4 * kPaThreads * kU) {
      int page[kU];
      float4 w[kU];
      int4 x[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int s = base + u * 4 * kPaThreads;
        page[u] = s < s1 ? page_of(p.c, b, s >> p.c.page_shift, p.status, DBG_PAGED_APPEND, 1) : -1;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t at = meta_at(max(page[u], 0), (base + u * 4 * kPaThreads) & page_mask);
        if (page[u] >= 0) {
          w[u] = *reinterpret_cast<const float4*>(p.c.weight + at);
          x[u] = *reinterpret_cast<const int4*>(p.c.pos + at);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int s = base + u * 4 * kPaThreads;
        const float wf[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        const int xi[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (s + i < s1) use(s + i, page[u] >= 0 ? key_of(wf[i], xi[i]) : kStays);
      }
    }
  };
  // Writes list entry `at`: token i of the sequence into `slot` (< 0: none for it).
  auto place = [&](int at, int i, int slot) {
    int page = -1, off = 0;
    int32_t out = -2;
    if (slot >= 0) {
      page = page_of(p.c, b, slot >> p.c.page_shift, p.status, DBG_PAGED_APPEND, 2);
      off = slot & page_mask;
    } else {
      debug_fail(p.status, DBG_PAGED_APPEND, 3);
    }
    if (page >= 0) {
      const int64_t to = meta_at(page, off);
      out = slot < n ? p.c.pos[to] : -1;
      p.c.pos[to] = seen + i;
      p.c.weight[to] = 0.f;
    }
    if (p.evicted != nullptr) p.evicted[static_cast<int64_t>(tok0 + i) * p.c.n_kv_heads + h] = out;
    l_page[at] = page;
    l_off[at] = off;
    l_tok[at] = tok0 + i;
  };
  auto copy = [&](int entries) {
    copy_rows<D, kF8, kPaThreads, 4>(p.c, p.k_new, p.v_new, p.token_stride, h, {l_page, l_off, l_tok}, entries);
  };

  if constexpr (!kChunk) {
    int slot = n;                                        // the free slot, if there is one
    if (e > 0) {
      uint64_t key = kStays;
      int at = -1;
      for_keys([&](int s, uint64_t k) {
        if (k < key) key = k, at = s;
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t k2 = __shfl_xor_sync(0xffffffffu, key, o);
        const int a2 = __shfl_xor_sync(0xffffffffu, at, o);
        if (k2 < key || (k2 == key && a2 < at)) key = k2, at = a2;
      }
      if (lane == 0) best_key[warp] = key, best_slot[warp] = at;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kPaWarps; ++w)
          if (best_key[w] < key || (best_key[w] == key && best_slot[w] < at)) key = best_key[w], at = best_slot[w];
        best_key[kPaWarps] = key;
        best_slot[kPaWarps] = at;
      }
      cluster.sync();
      key = kStays;
      slot = -1;
      for (int q = 0; q < ctas; ++q) {
        const uint64_t k2 = *cluster.map_shared_rank(&best_key[kPaWarps], q);
        const int a2 = *cluster.map_shared_rank(&best_slot[kPaWarps], q);
        if (k2 < key || (k2 == key && a2 < slot)) key = k2, slot = a2;
      }
    }
    cluster.sync();                                      // count and minima are read
    if (cta != 0) return;
    if (tid == 0) {
      place(0, 0, slot);
      p.c.count[row] = min(n + 1, cap);
      p.c.seen[row] = seen + 1;
    }
    __syncthreads();
    copy(1);
  } else {
    // Tokens for free slots, dealt to the cluster's CTAs in runs of kPaThreads.
    for (int base = cta * kPaThreads; base < f; base += ctas * kPaThreads) {
      const int k = min(kPaThreads, f - base);
      if (tid < k) place(tid, base + tid, n + base + tid);
      __syncthreads();
      copy(k);
      __syncthreads();
    }
    if (e > 0) {
      for_keys([&](int s, uint64_t k) { keys[s - s0] = k; });
      __syncthreads();
      // Radix select, smallest first.  A key with (key & mask) < prefix is taken, one with == prefix is undecided.
      uint64_t prefix = 0, mask = 0;
      uint32_t need = static_cast<uint32_t>(e);          // still to take among the undecided
      bool whole = false;                                // every undecided key is taken
      int pass = 0;
      for (int shift = 56; shift >= 0; shift -= 8, ++pass) {
        uint32_t* mine = hist[pass & 1];
        mine[tid] = 0;
        __syncthreads();
        for (int i = tid; i < s1 - s0; i += kPaThreads) {
          const uint64_t k = keys[i];
          if (k != kStays && (k & mask) == prefix) atomicAdd(&mine[(k >> shift) & 255u], 1u);
        }
        cluster.sync();        // a buffer is cleared again two passes on, past a barrier after its last reader
        uint32_t c = 0;
        for (int q = 0; q < ctas; ++q) c += cluster.map_shared_rank(mine, q)[tid];
        uint32_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[warp] = incl;
        if (tid == 0) sel[2] = 0;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += warp_sum[w];
        if (incl >= need && incl - c < need) {           // the digit that holds the need-th key
          sel[0] = tid;
          sel[1] = need - (incl - c);
          sel[2] = c == need - (incl - c) ? 2 : 1;
        }
        __syncthreads();
        const uint32_t state = sel[2];
        if (state == 0) {                                // fewer than need in all: take what there is
          whole = true;
          break;
        }
        prefix |= static_cast<uint64_t>(sel[0]) << shift;
        mask |= 255ull << shift;
        need = sel[1];
        __syncthreads();
        if (state == 2) {
          whole = true;
          break;
        }
      }
      // Victims of this slice: those below the prefix, and of the undecided all or (equal keys, which need equal
      // positions) the first `need` in slot order.
      uint32_t below = 0, equal = 0;
      for (int i = tid; i < s1 - s0; i += kPaThreads) {
        const uint64_t k = keys[i];
        if (k == kStays) continue;
        below += (k & mask) < prefix || (whole && (k & mask) == prefix);
        equal += !whole && (k & mask) == prefix;
      }
      uint32_t both = below | (equal << 16);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
      if (lane == 0) warp_sum[warp] = both;
      __syncthreads();
      if (tid == 0) {
        uint32_t all = 0;
        for (int w = 0; w < kPaWarps; ++w) all += warp_sum[w];
        taken_here = all;
      }
      cluster.sync();
      uint32_t rank = 0, all_taken = 0, seen_equal = 0, eq_all_before = 0;   // victims and undecided before this slice
      for (int q = 0; q < ctas; ++q) {
        const uint32_t x = *cluster.map_shared_rank(&taken_here, q);
        const uint32_t eq = x >> 16, left = need > eq_all_before ? need - eq_all_before : 0u;
        const uint32_t take = (x & 0xffffu) + min(eq, left);
        if (q == cta) seen_equal = eq_all_before;
        if (q < cta) rank += take;
        all_taken += take;
        eq_all_before += eq;
      }
      for (int base = s0; base < s1; base += kPaThreads) {
        const int s = base + tid;
        const uint64_t k = s < s1 ? keys[s - s0] : kStays;
        const bool eq = k != kStays && (k & mask) == prefix;
        const uint32_t eq_bits = __ballot_sync(0xffffffffu, eq && !whole);
        if (lane == 0) warp_sum[warp] = __popc(eq_bits);
        __syncthreads();
        uint32_t eq_rank = seen_equal + __popc(eq_bits & ((1u << lane) - 1u));
        uint32_t eq_all = 0;
        for (int w = 0; w < kPaWarps; ++w) {
          eq_rank += w < warp ? warp_sum[w] : 0u;
          eq_all += warp_sum[w];
        }
        const bool goes = k != kStays && ((k & mask) < prefix || (eq && (whole || eq_rank < need)));
        const uint32_t bits = __ballot_sync(0xffffffffu, goes);
        __syncthreads();
        if (lane == 0) warp_sum[warp] = __popc(bits);
        __syncthreads();
        uint32_t at = __popc(bits & ((1u << lane) - 1u)), all = 0;
        for (int w = 0; w < kPaWarps; ++w) {
          at += w < warp ? warp_sum[w] : 0u;
          all += warp_sum[w];
        }
        if (goes) place(at, f + rank + at, s);
        __syncthreads();
        copy(all);
        __syncthreads();
        rank += all;
        seen_equal += eq_all;
      }
      // Tokens for which no slot may be replaced.
      if (cta == 0)
        for (int i = f + all_taken + tid; i < m; i += kPaThreads) place(tid, i, -1);
    }
    cluster.sync();                                      // the cluster has read counts, histograms and sums
    if (cta == 0 && tid == 0) {
      p.c.count[row] = min(n + m, cap);
      p.c.seen[row] = seen + m;
    }
  }
}

// CTAs per row: the largest of 8, 4, 2, 1 whose clusters leave two CTAs per
// SM at most and 1,024 slots per CTA at least, but enough for the slice to fit.
cudaError_t launch_paged_append(PagedAppendParams& p, int head_dim, bool f8, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.c.batch) * p.c.n_kv_heads;
  int ctas = 8;
  while (ctas > 1 && (rows * ctas > 2 * 148 || p.c.capacity < 1024 * ctas)) ctas >>= 1;
  while (ctas < 8 && (p.c.capacity + ctas - 1) / ctas > kPaMaxSlice) ctas <<= 1;
  p.slice = ((p.c.capacity + ctas - 1) / ctas + 7) / 8 * 8;
  const bool chunk = !p.one_each;
  const size_t smem = chunk ? static_cast<size_t>(p.slice) * 8 : 0;
  const dim3 grid(static_cast<unsigned>(rows * ctas)), block(kPaThreads);
  static std::atomic<uint64_t> ready[4];
  auto go = [&](auto kern, int which) {
    if (smem > 0) {
      const cudaError_t e = allow_smem(kern, kPaMaxSlice * 8, ready[which]);
      if (e != cudaSuccess) return e;
    }
    return launch_paged(kern, grid, block, smem, ctas, stream, p);
  };
  if (head_dim == 128) {
    if (f8) return chunk ? go(paged_append_kernel<128, true, true>, 0) : go(paged_append_kernel<128, true, false>, 0);
    return chunk ? go(paged_append_kernel<128, false, true>, 1) : go(paged_append_kernel<128, false, false>, 1);
  }
  if (f8) return chunk ? go(paged_append_kernel<64, true, true>, 2) : go(paged_append_kernel<64, true, false>, 2);
  return chunk ? go(paged_append_kernel<64, false, true>, 3) : go(paged_append_kernel<64, false, false>, 3);
}

}  // namespace kvpop
