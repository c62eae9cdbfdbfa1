// Appending tokens to the paged cache, with eviction of the tokens of least
// accumulated attention weight, sm_100a.
//
// A row (sequence, KV head) is handled by a cluster of 1 to 8 CTAs, each of
// which looks at a slice of the row's slots.  Slots go in the order of their
// key, smaller = earlier: the order-preserving bits of the weight (NaN lowest),
// then, among equal weights, 2^31 - 1 - position; slots that may not go (sinks,
// recent tokens) have a key that no weight has.  One token in, one out (the
// steady state of decoding) is an argmin, bound by the bytes of weights and
// positions.  Several out is an exact radix select of the e-th smallest key
// over keys in shared memory, in digits of 11 bits (a weight's first digit is
// its exponent and two bits more, which spreads real weights over many
// counters): the cluster adds its histograms through distributed shared memory,
// and stops as soon as a digit's bucket is taken whole, mostly after two.
// Everything is integer, so the result is exact and depends on no order.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "kvpop_paged.cuh"

namespace kvpop {

namespace cg = cooperative_groups;

constexpr int kPaMaxSlice = 16384;     // keys one CTA holds at most (128 KiB); 8 x 16384 = the largest capacity
// Place of key i: the 8 words of 4 in a 128-byte line are permuted by the line's number, so that threads that each
// read consecutive keys meet different banks, and 4 keys stay together.
__device__ __forceinline__ int placed(int i) { return i ^ ((i >> 3) & 28); }
constexpr int kPaBits = 11;           // of a digit
constexpr int kPaBins = 1 << kPaBits;
constexpr int kPaList = kPaBins * 4 / static_cast<int>(sizeof(RowEntry));   // as the histogram
constexpr uint32_t kStays = ~0u;       // key of a slot that may not go; no weight has it

// Larger float -> larger key, never 2^32 - 1; -0 equals +0 (the addition makes it +0); NaN -> 0, below every number
// (the addition's NaN is the canonical 0x7fffffff, whose key 2^32 - 1 wraps to 0 with the one added to all).
__device__ __forceinline__ uint32_t weight_key(float f) {
  const uint32_t u = __float_as_uint(__fadd_rn(f, 0.f));
  return (u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u)) + 1u;
}

// The one of a warp's candidates that goes first: least key, then largest position, then smallest slot (at < 0: no
// candidate, with key ~0).  Every lane gets it.
struct Candidate {
  uint32_t key;
  int pos, at;
};
// Looks at four slots from s on, weights' bits w and positions x.  From +0 to +inf a weight's key is its bits plus
// 2^31 + 1; others take the long way.
__device__ __forceinline__ void consider(Candidate& c, const uint4& w, const int4& x, int s, uint32_t sinks, uint32_t span) {
  const uint32_t wu[4] = {w.x, w.y, w.z, w.w};
  const int xi[4] = {x.x, x.y, x.z, x.w};
  uint32_t k[4];
  if (max(max(w.x, w.y), max(w.z, w.w)) <= 0x7f800000u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = wu[e] + 0x80000001u;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = weight_key(__uint_as_float(wu[e]));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (static_cast<uint32_t>(xi[e]) - sinks >= span) k[e] = ~0u;       // with this key a candidate is none
    const bool better = (k[e] < c.key) | ((k[e] == c.key) & (xi[e] > c.pos));
    c.key = better ? k[e] : c.key;
    c.pos = better ? xi[e] : c.pos;
    c.at = better ? s + e : c.at;
  }
}
__device__ __forceinline__ Candidate first_to_go(const Candidate& c) {
  Candidate r;
  r.key = __reduce_min_sync(0xffffffffu, c.key);
  r.pos = __reduce_max_sync(0xffffffffu, c.key == r.key ? c.pos : -1);
  r.at = static_cast<int>(__reduce_min_sync(0xffffffffu, c.key == r.key && c.pos == r.pos ? static_cast<uint32_t>(c.at) : ~0u));
  return r;
}

// A warp writes token `tok` of the call, position `seen` of sequence b, into `slot` of row (b, h) (< 0: there is none
// for it), where position `old` goes (-1: nothing does); `fresh` is the lane's 16-byte word of its K row, then V's.
template <int D, bool kF8>
__device__ __forceinline__ void write_one(const PagedAppendParams& p, int b, int h, int tok, int slot, int old, int seen,
                                          const uint4& fresh) {
  const int lane = threadIdx.x & 31;
  const int off = slot & ((1 << p.c.page_shift) - 1);
  int page = -1;
  KVPOP_CHECK(slot < p.c.capacity && b < p.c.batch && h < p.c.n_kv_heads, p.dbg, DBG_PAGED_APPEND, 7);
  if (slot < 0) debug_fail(p.status, DBG_PAGED_APPEND, 3);
  else page = page_of(p.c, b, slot >> p.c.page_shift, p.status, DBG_PAGED_APPEND, 2);
  if (lane == 0 && p.evicted != nullptr) p.evicted[static_cast<int64_t>(tok) * p.c.n_kv_heads + h] = page >= 0 ? old : -2;
  if (page < 0) return;
  if (lane == 0) {
    const int64_t at = ((static_cast<int64_t>(page) * p.c.n_kv_heads + h) << p.c.page_shift) + off;
    p.c.pos[at] = seen;
    p.c.weight[at] = 0.f;
  }
  if (lane < D / 4) {
    const bool is_v = lane >= D / 8;
    const int word = lane % (D / 8);
    uint8_t* to = is_v ? p.c.v + page * p.c.v_page + h * p.c.v_head + off * p.c.v_slot
                       : p.c.k + page * p.c.k_page + h * p.c.k_head + off * p.c.k_slot;
    if constexpr (kF8) {
      const float* scale = is_v ? p.c.v_scale : p.c.k_scale;
      *reinterpret_cast<uint2*>(to + 8 * word) = to_e4m3x8(fresh, divisor_of(scale != nullptr ? scale[h] : 1.f));
    } else {
      *reinterpret_cast<uint4*>(to + 16 * word) = fresh;
    }
  }
}

template <int D, bool kF8, bool kChunk, int kPaThreads>
__global__ void __launch_bounds__(kPaThreads, 1024 / kPaThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int kPaWarps = kPaThreads / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  extern __shared__ __align__(16) uint32_t keys[];       // kChunk: weights' keys of this CTA's slice, then its positions
  __shared__ Candidate best[kPaWarps + 1];               // one out: of each warp; [kPaWarps] = of the CTA
  __shared__ __align__(16) uint32_t hist[kChunk ? kPaBins : 4];   // a pass's histogram, read by the cluster
  __shared__ uint32_t vary[2];                           // AND and OR of a pass's keys, read by the cluster
  __shared__ uint32_t every_any[2];                      // the same of the whole cluster
  __shared__ uint32_t sel[3];
  __shared__ uint32_t ranks[3];                          // victims before this slice, victims in all, undecided before it
  __shared__ uint32_t taken_here[2];                     // kChunk: victims and undecided in this slice, read by the cluster
  __shared__ uint32_t warp_sum[kPaWarps];

  // A barrier of the row's CTAs.
  auto sync_row = [&] {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / ctas, b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int page_mask = (1 << p.c.page_shift) - 1;
  const int tok0 = p.one_each ? b : p.start[b];
  const int m = p.one_each ? 1 : p.start[b + 1] - tok0;
  if (m == 0) return;                                    // as for every branch on b or count: the whole cluster
  grid_wait();
  grid_launch_next();
  // One out: a thread's slots are four at a time, kU times; their page numbers, and the new rows (a 16-byte word per
  // lane of warp 0), are on their way together with the row's counts.
  constexpr int kU = 4;
  const int s_lo = cta * p.slice;
  int raw[kU];
  uint4 fresh = make_uint4(0, 0, 0, 0);
  if constexpr (!kChunk) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = s_lo + 4 * (tid + u * kPaThreads);
      raw[u] = s < min(s_lo + p.slice, p.c.capacity) ? p.c.table[static_cast<int64_t>(b) * p.c.max_pages + (s >> p.c.page_shift)] : -1;
    }
    if (cta == 0 && tid < D / 4) {
      const uint16_t* from = (tid < D / 8 ? p.k_new : p.v_new) + tok0 * p.token_stride + static_cast<int64_t>(h) * D + 8 * (tid % (D / 8));
      fresh = *reinterpret_cast<const uint4*>(from);
    }
  }
  const int count = p.c.count[row], seen = p.c.seen[row];
  if (count < 0) {
    if (p.evicted != nullptr && cta == 0)
      for (int i = tid; i < m; i += kPaThreads) p.evicted[static_cast<int64_t>(tok0 + i) * p.c.n_kv_heads + h] = -2;
    return;
  }
  const int cap = p.c.capacity, n = min(count, cap), f = min(m, cap - n), e = m - f;
  // Tokens at positions sinks .. recent - 1 may go: recent is where the window begins once the new ones are in.  Smaller
  // positions less sinks wrap to numbers from 2^31 - sinks up, which no span exceeds.
  const int64_t recent = static_cast<int64_t>(seen) + m - p.window;
  const uint32_t span = static_cast<uint32_t>(max(int64_t(0), min(recent, int64_t(1) << 31) - p.sinks));
  const int s0 = min(n, cta * p.slice), s1 = min(n, s0 + p.slice);
  const uint16_t* k_src = p.k_new + tok0 * p.token_stride;
  const uint16_t* v_src = p.v_new + tok0 * p.token_stride;

  auto meta_at = [&](int page, int off) {
    return ((static_cast<int64_t>(page) * p.c.n_kv_heads + h) << p.c.page_shift) + off;
  };
  // Token i of the sequence into `slot` (< 0: none for it), where position `old` goes (-1: nothing does).
  auto place = [&](int i, int slot, int old) {
    int page = -1, off = 0;
    KVPOP_CHECK(i >= 0 && i < m && slot < cap, p.dbg, DBG_PAGED_APPEND, 6);
    if (slot >= 0) {
      page = page_of(p.c, b, slot >> p.c.page_shift, p.status, DBG_PAGED_APPEND, 2);
      off = slot & page_mask;
    } else {
      debug_fail(p.status, DBG_PAGED_APPEND, 3);
    }
    if (page >= 0) {
      const int64_t to = meta_at(page, off);
      p.c.pos[to] = seen + i;
      p.c.weight[to] = 0.f;
    }
    if (p.evicted != nullptr) p.evicted[static_cast<int64_t>(tok0 + i) * p.c.n_kv_heads + h] = page >= 0 ? old : -2;
    return row_entry(page, off, i);
  };

  if constexpr (!kChunk) {
    int slot = n, old = -1;                              // the free slot, if there is one
    if (e > 0) {
      Candidate c = {~0u, -1, -1};
      for (int base = s_lo + 4 * tid; base < s1; base += 4 * kPaThreads * kU) {
        uint4 w[kU];
        int4 x[kU];
        if (base != s_lo + 4 * tid)
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int s = base + u * 4 * kPaThreads;
            raw[u] = s < s1 ? p.c.table[static_cast<int64_t>(b) * p.c.max_pages + (s >> p.c.page_shift)] : -1;
          }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int s = base + u * 4 * kPaThreads;
          x[u] = make_int4(-1, -1, -1, -1);              // a position that never goes
          w[u] = make_uint4(0, 0, 0, 0);
          if (s < s1) {
            if (static_cast<uint32_t>(raw[u]) < static_cast<uint32_t>(p.c.n_pages)) {
              const int64_t from = meta_at(raw[u], s & page_mask);
              w[u] = *reinterpret_cast<const uint4*>(p.c.weight + from);
              x[u] = *reinterpret_cast<const int4*>(p.c.pos + from);
              if (s + 3 >= s1) {
                x[u].w = -1;
                if (s + 2 >= s1) x[u].z = -1;
                if (s + 1 >= s1) x[u].y = -1;
              }
            } else {
              debug_fail(p.status, DBG_PAGED_APPEND, 1);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) consider(c, w[u], x[u], base + u * 4 * kPaThreads, static_cast<uint32_t>(p.sinks), span);
      }
      c = first_to_go(c);
      if (lane == 0) best[warp] = c;
      __syncthreads();
      if (warp == 0) {
        c = lane < kPaWarps ? best[lane] : Candidate{~0u, -1, -1};
        c = first_to_go(c);
        if (lane == 0) best[kPaWarps] = c;
      }
      if (ctas > 1) {
        cluster.sync();
        if (cta == 0 && warp == 0) {
          c = lane < ctas ? *cluster.map_shared_rank(&best[kPaWarps], lane) : Candidate{~0u, -1, -1};
          c = first_to_go(c);
        }
      }
      slot = c.key == ~0u ? -1 : c.at;
      old = c.pos;
    }
    // Warp 0 of CTA 0 has the slot; every CTA's count and candidate has been read.
    sync_row();
    if (cta != 0) return;
    if (warp > 0) return;
    write_one<D, kF8>(p, b, h, tok0, slot, old, seen, fresh);
    if (lane == 0) {
      p.c.count[row] = min(n + 1, cap);
      p.c.seen[row] = seen + 1;
    }
  } else {
    // Rows to write, up to kPaList at a time, where the histogram is at other times.
    RowEntry* list = reinterpret_cast<RowEntry*>(hist);
    int32_t* spots = reinterpret_cast<int32_t*>(keys) + (p.slice + 31) / 32 * 32;
    // Tokens for free slots: an even share for each CTA of the cluster.
    if (f > 0) {
      const int share = (f + ctas - 1) / ctas, f0 = min(f, cta * share), f1 = min(f, f0 + share);
      for (int done = f0; done < f1; done += kPaList) {
        const int entries = min(f1 - done, kPaList);
        for (int i = tid; i < entries; i += kPaThreads) list[i] = place(done + i, n + done + i, -1);
        __syncthreads();
        copy_rows<D, kF8, kPaThreads, 8>(p.c, k_src, v_src, p.token_stride, h, list, entries);
        __syncthreads();
      }
    }
    if (e > 0) {
      // Radix select, smallest first, over the weights' keys and, where equal weights leave a choice, over the
      // positions' among those.  A key with (key & mask) < prefix is taken, one with == prefix is undecided.  Each
      // pass counts a digit and also finds which bits vary among the undecided keys, so that the next digit starts at
      // the first one that does: keys that are all equal cost one pass, not three.  The first pass counts while the
      // keys arrive.
      uint32_t need = static_cast<uint32_t>(e);          // still to take among the undecided
      auto clear = [&] {
        for (int i = tid; i < kPaBins / 4; i += kPaThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) sel[2] = 0, vary[0] = ~0u, vary[1] = 0u;
        __syncthreads();
      };
      // Counters that many keys share would serialise the lanes: one addition for those that agree with lane 0's key.
      auto count = [&](bool in, uint32_t digit) {
        const uint32_t first = __shfl_sync(0xffffffffu, digit, 0);
        const bool same = in && digit == first;
        const uint32_t votes = __ballot_sync(0xffffffffu, same);
        if (lane == 0 && votes != 0) atomicAdd(&hist[first], static_cast<uint32_t>(__popc(votes)));
        if (in && !same) atomicAdd(&hist[digit], 1u);
      };
      uint32_t every = ~0u, any = 0;                     // AND and OR of the undecided keys
      clear();
      for (int base = s0; base < s1; base += 4 * kPaThreads * kU) {
        int page[kU];
        float4 w[kU];
        int4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int s = base + 4 * (tid + u * kPaThreads);
          page[u] = s < s1 ? page_of(p.c, b, s >> p.c.page_shift, p.status, DBG_PAGED_APPEND, 1) : -1;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int s = base + 4 * (tid + u * kPaThreads);
          const int64_t at = meta_at(max(page[u], 0), s & page_mask);
          w[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          x[u] = make_int4(-1, -1, -1, -1);              // a position that never goes
          if (page[u] >= 0) {
            w[u] = *reinterpret_cast<const float4*>(p.c.weight + at);
            x[u] = *reinterpret_cast<const int4*>(p.c.pos + at);
            if (s + 3 >= s1) {
              x[u].w = -1;
              if (s + 2 >= s1) x[u].z = -1;
              if (s + 1 >= s1) x[u].y = -1;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = base - s0 + 4 * (tid + u * kPaThreads);
          const float wf[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
          const int xi[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t k[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool in = static_cast<uint32_t>(xi[j]) - static_cast<uint32_t>(p.sinks) < span;
            k[j] = in ? weight_key(wf[j]) : kStays;
            if (in) every &= k[j], any |= k[j];
            count(in, k[j] >> (32 - kPaBits));
          }
          // Slices end at multiples of 8, rows need not: the words past s1 hold keys that stay.
          if (i < p.slice && KVPOP_IN(i + 4 <= p.slice, p.dbg, DBG_PAGED_APPEND, 4)) {
            *reinterpret_cast<uint4*>(&keys[placed(i)]) = make_uint4(k[0], k[1], k[2], k[3]);
            *reinterpret_cast<int4*>(&spots[placed(i)]) = x[u];
          }
        }
      }
      const int here_n = s1 - s0;
      uint32_t prefix = 0, mask = 0, tied = 0;           // tied: the weights' key whose positions decide
      bool whole = false, ties = false;                  // every undecided key is taken; positions decide
      for (int pass = 0, top = 32;; ++pass) {            // bits top .. 31 are decided
        if (top == 0) {
          if (ties) break;                               // equal weights and positions: the first `need` in slot order
          ties = true;
          tied = prefix;
          // Positions that may go are below `recent`: 2^31 - 1 less one of them has ones from their bits up to bit 30.
          top = 32 - __clz(static_cast<int>(static_cast<uint32_t>(min(recent, int64_t(1) << 31) - 1) & 0x7fffffffu));
          mask = ~((1u << top) - 1u);
          prefix = 0x7fffffffu & mask;
          if (top == 0) break;                           // only position 0 may go
        }
        const int bits = min(top, kPaBits), shift = top - bits;
        if (pass > 0) {
          sync_row();          // every CTA has read this one's counters
          clear();
          every = ~0u, any = 0;
          for (int base = 0; base < here_n; base += kPaThreads) {
            const int i = base + tid;
            uint32_t k = i < here_n ? keys[placed(i)] : kStays;
            bool in = k != kStays;
            if (ties) {
              in = k == tied;
              if (in) k = 0x7fffffffu - static_cast<uint32_t>(spots[placed(i)]);
            }
            in = in && (k & mask) == prefix;
            if (__ballot_sync(0xffffffffu, in) == 0) continue;
            if (in) every &= k, any |= k;
            count(in, (k >> shift) & ((1u << bits) - 1));
          }
        }
        {
          const uint32_t a1 = __reduce_and_sync(0xffffffffu, every), o1 = __reduce_or_sync(0xffffffffu, any);
          if (lane == 0) {
            atomicAnd(&vary[0], a1);
            atomicOr(&vary[1], o1);
          }
        }
        sync_row();
        constexpr int kPer = kPaBins / kPaThreads;       // consecutive counters of a thread
        uint32_t c[kPer] = {}, all = 0;
#pragma unroll
        for (int j = 0; j < kPer / 4; ++j) {
          const int at = tid * (kPer / 4) + j;
          if (ctas == 1) {
            const uint4 x = reinterpret_cast<const uint4*>(hist)[at];
            c[4 * j] = x.x, c[4 * j + 1] = x.y, c[4 * j + 2] = x.z, c[4 * j + 3] = x.w;
            continue;
          }
#pragma unroll
          for (int q0 = 0; q0 < 8; q0 += 4) {            // four peers' words on their way at a time
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = make_uint4(0, 0, 0, 0);
              if (q0 + i < ctas) x[i] = reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, q0 + i))[at];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) c[4 * j] += x[i].x, c[4 * j + 1] += x[i].y, c[4 * j + 2] += x[i].z, c[4 * j + 3] += x[i].w;
          }
        }
        if (warp == 0) {
          uint32_t v0 = ~0u, v1 = 0u;
          if (lane < ctas) {
            const uint32_t* v = cluster.map_shared_rank(vary, lane);
            v0 = v[0], v1 = v[1];
          }
          v0 = __reduce_and_sync(0xffffffffu, v0);
          v1 = __reduce_or_sync(0xffffffffu, v1);
          if (lane == 0) every_any[0] = v0, every_any[1] = v1;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) all += c[i];
        uint32_t incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += warp_sum[w];
        if (incl >= need && incl - all < need) {         // this thread's counters hold the need-th key
          uint32_t before = incl - all, digit = 0, size = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (size == 0) {
              if (before + c[i] >= need) digit = tid * kPer + i, size = c[i];
              else before += c[i];
            }
          sel[0] = digit;
          sel[1] = need - before;
          sel[2] = size == need - before ? 2 : 1;
        }
        __syncthreads();
        const uint32_t state = sel[2];
        if (state == 0) {                                // fewer than need in all: take what there is
          whole = true;
          break;
        }
        prefix |= sel[0] << shift;
        mask |= ((1u << bits) - 1) << shift;
        need = sel[1];
        if (state == 2) {
          whole = true;
          break;
        }
        // The undecided keys agree in every bit from `shift` up now; of those below, skip the ones in which not even
        // this pass's keys differed.
        const uint32_t low = (1u << shift) - 1u, differ = (every_any[0] ^ every_any[1]) & low;
        top = 32 - __clz(static_cast<int>(differ));
        const uint32_t agreed = low & ~(top == 32 ? ~0u : (1u << top) - 1u);
        prefix |= every_any[0] & agreed;
        mask |= agreed;
        __syncthreads();                                 // the shared words of this pass are read
      }
      // Victims of this slice: those below the prefix, and of the undecided all or (equal keys and positions) the
      // first `need` in slot order.  A thread looks at `per` consecutive slots and remembers what it saw in a bit each.
      const int per = (p.slice + kPaThreads - 1) / kPaThreads;         // <= 32: the host gives long slices more threads
      const int i0 = tid * per, in_thread = max(0, min(per, here_n - i0));
      uint32_t below_bits = 0, equal_bits = 0;
      if (!ties) {
        const uint32_t last = min(prefix | ~mask, kStays - 1u);        // the largest key that is taken
        for (int j = 0; j < in_thread; ++j) below_bits |= static_cast<uint32_t>(keys[placed(i0 + j)] <= last) << j;
      } else {
        for (int j = 0; j < in_thread; ++j) {
          const uint32_t k = keys[placed(i0 + j)];
          below_bits |= static_cast<uint32_t>(k < tied) << j;
          if (k != tied) continue;
          const uint32_t head = (0x7fffffffu - static_cast<uint32_t>(spots[placed(i0 + j)])) & mask;
          below_bits |= static_cast<uint32_t>(head < prefix || (whole && head == prefix)) << j;
          equal_bits |= static_cast<uint32_t>(!whole && head == prefix) << j;
        }
      }
      // Exclusive scans over the block, below and equal in a word (at most 1,024 of each in a warp), and the totals.
      const uint32_t own = __popc(below_bits) | (__popc(equal_bits) << 16);
      uint32_t both = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, both, o);
        if (lane >= o) both += y;
      }
      if (lane == 31) warp_sum[warp] = both;
      __syncthreads();
      uint32_t below = (both - own) & 0xffffu, equal = (both - own) >> 16, below_all = 0, equal_all = 0;
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) {
        const uint32_t x = warp_sum[w];
        below_all += x & 0xffffu, equal_all += x >> 16;
        if (w < warp) below += x & 0xffffu, equal += x >> 16;
      }
      if (tid == 0) taken_here[0] = below_all, taken_here[1] = equal_all;
      sync_row();
      if (warp == 0) {
        // Lane q holds slice q's counts; undecided keys are taken in slice order until `need` are.
        uint32_t bel = 0, eq = 0;
        if (lane < ctas) {
          const uint32_t* x = cluster.map_shared_rank(taken_here, lane);
          bel = x[0], eq = x[1];
        }
        uint32_t eq_incl = eq;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, eq_incl, o);
          if (lane >= o) eq_incl += y;
        }
        const uint32_t eq_excl = eq_incl - eq;
        const uint32_t take = bel + min(eq, need > eq_excl ? need - eq_excl : 0u);
        uint32_t incl = take;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == cta) ranks[0] = incl - take, ranks[2] = eq_excl;
        if (lane == 7) ranks[1] = incl;
      }
      __syncthreads();
      const uint32_t rank0 = ranks[0], all_taken = ranks[1], seen_equal = ranks[2];
      const uint32_t left = need > seen_equal ? need - seen_equal : 0u;     // undecided ones that this slice gives
      uint32_t goes = below_bits;
      if (equal_bits != 0) {
        uint32_t eq_rank = equal;
        for (uint32_t bits = equal_bits; bits != 0; bits &= bits - 1, ++eq_rank)
          if (eq_rank < left) goes |= bits & (0u - bits);
      }
      const int here = static_cast<int>(below_all + min(equal_all, left));
      const uint32_t first = below + min(equal, left);                      // rank of this thread's first victim
      for (int done = 0; done < here; done += kPaList) {
        // Slots and positions in slot order, then a row entry for each.
        uint32_t at = first - static_cast<uint32_t>(done);                  // wraps: outside the list
        for (uint32_t bits = goes; bits != 0; bits &= bits - 1, ++at) {
          const int i = i0 + __ffs(bits) - 1;
          if (at < kPaList && KVPOP_IN(s0 + i < n, p.dbg, DBG_PAGED_APPEND, 5))
            list[at] = {s0 + i, static_cast<uint32_t>(spots[placed(i)])};
        }
        __syncthreads();
        const int entries = min(here - done, kPaList);
        for (int i = tid; i < entries; i += kPaThreads)
          list[i] = place(f + static_cast<int>(rank0) + done + i, list[i].page, static_cast<int>(list[i].off_tok));
        __syncthreads();
        copy_rows<D, kF8, kPaThreads, 8>(p.c, k_src, v_src, p.token_stride, h, list, entries);
        __syncthreads();
      }
      // Tokens for which no slot may be replaced.
      if (cta == 0)
        for (int i = f + static_cast<int>(all_taken) + tid; i < m; i += kPaThreads) place(i, -1, -2);
    }
    sync_row();                                      // the cluster has read counts, histograms and sums
    if (cta == 0 && tid == 0) {
      p.c.count[row] = min(n + m, cap);
      p.c.seen[row] = seen + m;
    }
  }
}

// One token into each of many rows: the argmin of paged_append_kernel as a
// stream.  A CTA takes every gridDim.x-th row in steps of kPsSlots slots; while
// it looks at one step's weights and positions, the next one's, and the page
// numbers, counts and new rows of the one after that, are on their way into
// shared memory, so the SM always has bytes in flight and no load is waited for
// (256 x 8 rows of 4,032 slots: 23.9 us with a CTA per row, 19.5 so).
// A thread reads what it copied itself; the barrier of a row's end shows warp 0
// the rest.
constexpr int kPsThreads = 256;
constexpr int kPsWarps = kPsThreads / 32;
constexpr int kPsU = 4;                                   // 16-byte words of weights (and positions) of a thread
constexpr int kPsSlots = 4 * kPsThreads * kPsU;

struct StreamSmem {
  uint4 words[2][2][kPsU][kPsThreads];                    // [step parity][weights, positions]
  int32_t pages[2][kPsU][kPsThreads];
  int32_t row[3][kPsWarps][2];                            // count and seen, a copy per warp
  uint4 fresh[3][32];                                     // the new K and V row, for warp 0
  Candidate best[2][kPsWarps];
};

__device__ __forceinline__ void copy16_to(void* smem, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(p)
               : "memory");
}
__device__ __forceinline__ void copy4_to(void* smem, const void* p) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(p)
               : "memory");
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kPsThreads, 3) paged_append_stream_kernel(const __grid_constant__ PagedAppendParams p) {
  extern __shared__ __align__(16) uint8_t stream_smem[];
  StreamSmem& sm = *reinterpret_cast<StreamSmem*>(stream_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = p.c.n_kv_heads, rows = p.c.batch * heads, cap = p.c.capacity;
  const int steps = (cap + kPsSlots - 1) / kPsSlots;      // of a row
  const int page_mask = (1 << p.c.page_shift) - 1;
  grid_wait();
  grid_launch_next();

  // A step of a row, and the ones after it.
  struct Step {
    int row, b, h, part;
  };
  auto advance = [&](Step& u) {
    if (++u.part < steps) return;
    u.part = 0;
    u.row += gridDim.x;
    u.b = u.row / heads;
    u.h = u.row - u.b * heads;
  };
  // Pages and counts, and with a row's last step its new rows.
  auto ask_meta = [&](const Step& u, int at, int parity) {
    if (u.row >= rows) return;
    const int32_t* table = p.c.table + static_cast<int64_t>(u.b) * p.c.max_pages;
#pragma unroll
    for (int i = 0; i < kPsU; ++i) {
      const int s = u.part * kPsSlots + 4 * (tid + i * kPsThreads);
      if (s < cap) copy4_to(&sm.pages[parity][i][tid], table + (s >> p.c.page_shift));
    }
    if (lane < 2) copy4_to(&sm.row[at][warp][lane], (lane == 0 ? p.c.count : p.c.seen) + u.row);
    if (warp == 0 && lane < D / 4 && u.part == steps - 1) {
      const uint16_t* from = (lane < D / 8 ? p.k_new : p.v_new) + u.b * p.token_stride + static_cast<int64_t>(u.h) * D + 8 * (lane % (D / 8));
      copy16_to(&sm.fresh[at][lane], from);
    }
  };
  auto meta_at = [&](int page, int h, int off) {
    return ((static_cast<int64_t>(page) * heads + h) << p.c.page_shift) + off;
  };
  // Words that a step has to look at, a bit each: none while the row has a free slot, or takes no part.
  auto ask_words = [&](const Step& u, int at, int parity) {
    int here = 0;
    if (u.row >= rows || sm.row[at][warp][0] < cap) return here;
#pragma unroll
    for (int i = 0; i < kPsU; ++i) {
      const int s = u.part * kPsSlots + 4 * (tid + i * kPsThreads);
      if (s >= cap) continue;
      const int page = sm.pages[parity][i][tid];
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.n_pages)) {
        debug_fail(p.status, DBG_PAGED_APPEND, 1);
        continue;
      }
      const int64_t from = meta_at(page, u.h, s & page_mask);
      copy16_to(&sm.words[parity][0][i][tid], p.c.weight + from);
      copy16_to(&sm.words[parity][1][i][tid], p.c.pos + from);
      here |= 1 << i;
    }
    return here;
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  auto landed = [] {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();                                         // count and seen are two lanes' copies
  };

  Step now = {static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.x) / heads, static_cast<int>(blockIdx.x) % heads, 0};
  Step next = now;
  advance(next);
  ask_meta(now, 0, 0);
  commit();
  landed();
  int here = ask_words(now, 0, 0);
  ask_meta(next, 1, 1);
  commit();
  Candidate c = {~0u, -1, -1};
  int at = 0, parity = 0, best_at = 0;                    // of the step at hand
  while (now.row < rows) {
    landed();                                             // this step's words, the next one's pages and counts
    Step after = next;
    if (next.row < rows) advance(after);
    const int at1 = at == 2 ? 0 : at + 1, at2 = at1 == 2 ? 0 : at1 + 1;
    const int here_next = ask_words(next, at1, parity ^ 1);
    ask_meta(after, at2, parity);                         // this step's pages are done with
    commit();
    const int count = sm.row[at][warp][0], seen = sm.row[at][warp][1];
    if (count >= cap) {
      const int64_t recent = static_cast<int64_t>(seen) + 1 - p.window;
      const uint32_t span = static_cast<uint32_t>(max(int64_t(0), min(recent, int64_t(1) << 31) - p.sinks));
#pragma unroll
      for (int i = 0; i < kPsU; ++i) {
        if (((here >> i) & 1) == 0) continue;
        const int s = now.part * kPsSlots + 4 * (tid + i * kPsThreads);
        const uint4 w = sm.words[parity][0][i][tid];
        int4 x = *reinterpret_cast<const int4*>(&sm.words[parity][1][i][tid]);
        if (s + 3 >= cap) {
          x.w = -1;
          if (s + 2 >= cap) x.z = -1;
          if (s + 1 >= cap) x.y = -1;
        }
        consider(c, w, x, s, static_cast<uint32_t>(p.sinks), span);
      }
    }
    if (now.part == steps - 1) {                          // the row's last step
      c = first_to_go(c);
      if (lane == 0) sm.best[best_at][warp] = c;
      __syncthreads();
      if (warp == 0) {
        c = lane < kPsWarps ? sm.best[best_at][lane] : Candidate{~0u, -1, -1};
        c = first_to_go(c);
        if (count < 0) {
          if (lane == 0 && p.evicted != nullptr) p.evicted[static_cast<int64_t>(now.b) * heads + now.h] = -2;
        } else {
          const int slot = count < cap ? count : c.key == ~0u ? -1 : c.at;
          write_one<D, kF8>(p, now.b, now.h, now.b, slot, count < cap ? -1 : c.pos, seen, sm.fresh[at][lane]);
          if (lane == 0) {
            p.c.count[now.row] = min(count, cap - 1) + 1;        // count may be any int32
            p.c.seen[now.row] = seen + 1;
          }
        }
      }
      c = {~0u, -1, -1};
      best_at ^= 1;                                       // its other buffer was read before the last barrier
    }
    now = next;
    next = after;
    here = here_next;
    at = at1;
    parity ^= 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

constexpr int kPsRows = 3 * 148;     // more rows than this are streamed

// CTAs per row.  One out: the largest of 8, 4, 2, 1 that leaves 1,024 slots per
// CTA at least, and two CTAs per SM at most or 8,192 slots per CTA (16 x 5
// rows of 96,250 slots: 26 us with 8 CTAs per row, 39 with 2).  Several out:
// the fewest that leave slices of 8,192 slots at most (12,800 for many rows,
// rather than 4 CTAs per row: 86 x 4 rows of 23,581 slots 85 and 109 us), and
// more while half the SMs would have no CTA and slices are over 2,048 slots:
// every pass of the select is a barrier of the cluster, and larger clusters
// wait for room (24 x 8 rows of 16,000 slots: 47, 41, 56 and 121 us with 1, 2,
// 4 and 8 CTAs per row, since then 38 with 2; 4 x 8 rows: 35, 23 and 33 us with
// 1, 4 and 8).  Three CTAs per SM of 512 or 384 threads took 44 to 52 us for the
// 24 x 8 rows when two took 38.
cudaError_t launch_paged_append(PagedAppendParams& p, int head_dim, bool f8, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.c.batch) * p.c.n_kv_heads;
  const bool chunk = !p.one_each;
  if (!chunk && rows > kPsRows) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(rows, 3 * 148))), block(kPsThreads);
    constexpr size_t kPsSmem = sizeof(StreamSmem);
    static SmemReady ready[4];
    auto go = [&](auto kern, int which) {
      const cudaError_t e = allow_smem(kern, kPsSmem, ready[which]);
      return e != cudaSuccess ? e : launch_paged(kern, grid, block, kPsSmem, 1, stream, p);
    };
    if (head_dim == 128)
      return f8 ? go(paged_append_stream_kernel<128, true>, 0) : go(paged_append_stream_kernel<128, false>, 1);
    return f8 ? go(paged_append_stream_kernel<64, true>, 2) : go(paged_append_stream_kernel<64, false>, 3);
  }
  int ctas = 1;
  if (chunk) {
    const int most = p.c.capacity > 2 * 8192 && rows * 4 > 2 * 148 ? 12800 : 8192;      // at 12,800 two still share an SM
    while (ctas < 8 && (p.c.capacity > most * ctas || (rows * ctas <= 74 && p.c.capacity > 2048 * ctas))) ctas <<= 1;
  } else {
    ctas = 8;
    while (ctas > 1 && (p.c.capacity < 1024 * ctas || (rows * ctas > 2 * 148 && p.c.capacity < 8192 * ctas))) ctas >>= 1;
  }
  p.slice = ((p.c.capacity + ctas - 1) / ctas + 7) / 8 * 8;
  // Many short slices take 256 threads, so that four CTAs share an SM (200 x 8 rows of 1,000 slots: 65 us, with 512
  // threads 87; 8 rows of 16,000 slots: 15 and 13).
  const bool small = !chunk || (p.slice <= 4096 && rows * ctas > 2 * 148);
  const size_t smem = chunk ? static_cast<size_t>(p.slice + 31) / 32 * 256 : 0;
  const dim3 grid(static_cast<unsigned>(rows * ctas)), block(small ? 256 : 512);
  static SmemReady ready[8];
  auto go = [&](auto kern, int which) {
    if (smem > 0) {
      const cudaError_t e = allow_smem(kern, kPaMaxSlice * 8, ready[which]);
      if (e != cudaSuccess) return e;
    }
    return launch_paged(kern, grid, block, smem, ctas, stream, p);
  };
  auto of = [&](auto dim, auto eight, int which) {
    constexpr int D = decltype(dim)::value;
    constexpr bool kF8 = decltype(eight)::value;
    if (!chunk) return go(paged_append_kernel<D, kF8, false, 256>, which);
    return small ? go(paged_append_kernel<D, kF8, true, 256>, which) : go(paged_append_kernel<D, kF8, true, 512>, which + 1);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (head_dim == 128) return f8 ? of(D128(), std::true_type(), 0) : of(D128(), std::false_type(), 2);
  return f8 ? of(D64(), std::true_type(), 4) : of(D64(), std::false_type(), 6);
}

}  // namespace kvpop
