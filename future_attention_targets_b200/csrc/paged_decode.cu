// One decode step of attention over the paged cache, sm_100a.
//
//   s[g, c] = scale q[g] . K[c]     lse[g] = ln sum_c exp(s[g, c])
//   out[g]  = sum_c exp(s[g, c] - lse[g]) V[c]
//   weight[c] += sum_g exp(s[g, c] - lse[g])                (optional)
//
// K and V are read once and every byte of them takes part in 2 G to 4 G
// multiply-adds, far below what the tensor pipe could do per byte: the bound
// is the HBM, and what counts is bytes in flight.  So each warp keeps a ring
// of tiles of 16 slots in shared memory, filled by 16-byte asynchronous copies
// several tiles ahead of the one it computes, with no barrier between warps;
// since every 8 slots compute their own address, a page may lie anywhere and
// rows may have any stride.
//
// The fragments of mma.m16n8k16 are read with plain 16-byte loads, because
// the product does not care in which order its inner indexes run:
//   K  is the B operand (n = key, k = head dim).  Lane (g, t) of the warp
//      (g = lane / 4, t = lane % 4) reads 16 bytes of row g at chunk t + 4 j;
//      the chunk's elements serve as its k indexes, and q is fetched in the
//      same order.
//   V  is the B operand of the second product (k = slot, n = head dim).  Lane
//      (g, t) reads 16 bytes of rows 2t, 2t + 1, 2t + 8, 2t + 9 at chunk g; a
//      byte permute pairs the two rows of a k pair, and n runs over the head
//      dim in whatever order the chunks give.
// Chunk c of row r lies at c ^ (r & 6) ^ 4 (r & 1): both patterns touch every
// bank once per 8 lanes.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "kvpop_paged.cuh"

namespace kvpop {

namespace cg = cooperative_groups;

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdMaxSplit = 2048;           // slots of one CTA at most
constexpr int kPdMinPage = 8;
constexpr int kPdMaxCluster = 16;
constexpr float kLn2 = 0.6931471805599453f;

// K and V pass through the L2 once: they are the first to leave it, so that the scores written meanwhile are still
// there for the second kernel.
__device__ __forceinline__ uint64_t passing() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ uint64_t staying() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void store_staying(float* p, float a, float b, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v2.f32 [%0], {%1, %2}, %3;" ::"l"(p), "f"(a), "f"(b), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t smem, const uint8_t* p, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2;" ::"r"(smem), "l"(p), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A B, 16 x 8 x 16, fp32 accumulation; bf16 operands, or fp16 for an 8-bit cache.
template <bool kF8>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (kF8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Two e4m3 values to two fp16 ones: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t v;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"(static_cast<uint16_t>(two)));
  return v;
}
// A pair of probabilities as a high part in the operand type and the rest as
// a low one: 16 bits of mantissa in bf16, 22 in fp16, so the products with V,
// which are exact in fp32, see the probability to 2^-17 or better.
template <bool kF8>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  if constexpr (kF8) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(a - bf_lo(hi), b - bf_hi(hi));
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}

// A tile in shared memory: K rows, then V rows.  Rows of 256 bytes come 16 at a
// time, shorter ones 32: a step's chain of products, maximum, exponentials and
// products costs about the same either way, and an e4m3 cache with half the
// bytes per slot was bound by that chain (32 x 8 x 8,192 slots: 66.8 us with
// 16, (see below) us with 32).
template <int D, bool kF8>
struct Tile {
  static constexpr int kRow = D * (kF8 ? 1 : 2);                // bytes of a slot's K (or V)
  static constexpr int kChunks = kRow / 16;
  static constexpr int kSlots = kRow == 256 ? 16 : 32;
  static constexpr int kH = kSlots / 8;                         // groups of 8 slots, each on one page
  static constexpr int kBytes = 2 * kSlots * kRow;
  static constexpr int kK = kRow / 64;                          // 16-byte chunks of a K row per lane
  static constexpr int kV = kRow >= 128 ? kRow / 128 : 1;       // 16-byte (8-byte when a row is 64) chunks of a V row
  // Two CTAs per SM with rings of 3 tiles where the registers allow no more, else three with 2 (4 short ones): the
  // chain of a step is then hidden by more warps (96 x 4 e4m3 rows of 8,192 slots, no weights: 178 -> 161 us).
  static constexpr int kStages = kRow == 64 ? 4 : kRow == 128 ? 2 : 3;
  static constexpr int ctas(bool wide) { return wide || kRow == 256 ? 2 : 3; }
  static constexpr int kRing = kStages * kBytes;                // bytes of a warp's ring
};

// Chunk permutation of row r within a tile.
__device__ __forceinline__ int swizzle(int r) { return (r & 6) ^ ((r & 1) << 2); }

// kWide: 9 to 16 query heads per CTA, else up to 8.  With up to 8 heads the
// lower 8 rows of the 16-row A operand are free, and the second product puts
// the low parts of the probabilities there: both parts in one instruction.
template <int D, bool kF8, bool kWide>
__global__ void __launch_bounds__(kPdThreads, Tile<D, kF8>::ctas(kWide)) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  using T = Tile<D, kF8>;
  constexpr int NT = D / 8;                 // 8-column tiles of out
  constexpr int KS = D / 16;                // k steps of q . K
  constexpr int kRows = kWide ? 16 : 8;     // query heads a CTA holds
  constexpr float kShift = kF8 ? 8.f : 0.f; // probabilities are held times 2^kShift: fp16's small end stays out of the way
  __shared__ int32_t pages[kPdMaxSplit / kPdMinPage + 1];
  __shared__ float sm_m[kPdWarps][kRows], sm_l[kPdWarps][kRows];
  extern __shared__ __align__(128) uint8_t rings[];
  float (*sm_o)[kRows][D] = reinterpret_cast<float (*)[kRows][D]>(rings);   // once the rings are done with
  static_assert(kRows * D * 4 <= T::kRing, "the warps' outputs reuse their rings");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  // A row's splits are a cluster, or (p.cluster == 0) CTAs of their own whose parts a second kernel joins.
  const int item = p.cluster ? blockIdx.x / p.n_split : blockIdx.x;
  const int split = p.cluster ? blockIdx.x % p.n_split : blockIdx.y;
  const int hc = item % p.head_chunks;                    // chunk of 16 heads of the group
  const int row = item / p.head_chunks;                   // (b, h)
  const int b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int G = min(p.group - hc * 16, 16);               // query heads of this CTA
  const int64_t bg0 = static_cast<int64_t>(b) * p.n_q_heads + h * p.group + hc * 16;
  const int lo = split * p.split_slots;

  grid_wait();
  // The pages of the range's slots are on their way while the row's count is; only those in use are looked at below.
  const int count = p.c.count[row];
  const int e0 = lo >> p.c.page_shift;
  const int ents = ((min(lo + p.split_slots, p.c.capacity) - 1) >> p.c.page_shift) - e0 + 1;
  for (int i = threadIdx.x; i < ents; i += kPdThreads) pages[i] = p.c.table[static_cast<int64_t>(b) * p.c.max_pages + e0 + i];
  const int n = min(max(count, 0), p.c.capacity);
  const int cnt = min(n - lo, p.split_slots);             // slots of this CTA
  // Splits with slots: those of a cluster wait for one another, the rest are gone by then (a barrier of the cluster
  // does not wait for threads that have exited).
  const int active = min(p.n_split, (n + p.split_slots - 1) / p.split_slots);
  if (cnt <= 0) {
    grid_launch_next();
    if (!p.cluster)
      for (int i = threadIdx.x; i < G; i += kPdThreads) p.part_ml[(bg0 + i) * p.n_split + split] = make_float2(-INFINITY, 0.f);
    if (p.cluster && split == 0) {                        // n = 0
      for (int i = threadIdx.x; i < G * D; i += kPdThreads) p.out[bg0 * D + i] = 0;
      if (p.lse != nullptr)
        for (int i = threadIdx.x; i < G; i += kPdThreads) p.lse[bg0 + i] = -INFINITY;
    }
    return;
  }
  // A page that the pool does not have is -1 from here on.
  for (int i = threadIdx.x; i <= ((lo + cnt - 1) >> p.c.page_shift) - e0; i += kPdThreads)
    if (static_cast<uint32_t>(pages[i]) >= static_cast<uint32_t>(p.c.n_pages)) {
      pages[i] = -1;
      debug_fail(p.status, DBG_PAGED_DECODE, 1);
    }

  // q in the order of K's chunks: A operand rows g and (wide) g + 8.
  uint32_t qa[KS][kWide ? 4 : 2];
  float qs[kWide ? 2 : 1];                                // score per unit of product, log2 units
#pragma unroll
  for (int r = 0; r < (kWide ? 2 : 1); ++r) {
    const int head = g + 8 * r;
    const uint16_t* qr = p.q + b * p.q_stride + static_cast<int64_t>(h * p.group + hc * 16 + head) * D;
    uint32_t x[KS][2];                                    // bf16 pairs: k step s, first and second half
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      // bf16 cache: chunk j holds dims 32 j + 8 t + 0..7, two k steps; e4m3: dims 64 j' + 16 t + 0..15, four.
      const int d0 = kF8 ? 64 * (j / 2) + 16 * t + 8 * (j & 1) : 32 * j + 8 * t;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (head < G) w = __ldg(reinterpret_cast<const uint4*>(qr + d0));
      x[2 * j][0] = w.x, x[2 * j][1] = w.y, x[2 * j + 1][0] = w.z, x[2 * j + 1][1] = w.w;
    }
    qs[r] = p.scale_log2;
    if constexpr (kF8) {
      // fp16 q: scaled by a power of two so that its largest entry is in [1/2, 1): exact for every entry down
      // to 2^-14 of it, and to 2^-25 of it below.
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) top = fmaxf(top, fmaxf(fabsf(bf_lo(x[s][i])), fabsf(bf_hi(x[s][i]))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = 0;
      if (top > 0.f && top < INFINITY) frexpf(top, &e);
      e = max(-120, min(120, e));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      qs[r] *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (p.c.k_scale != nullptr ? p.c.k_scale[h] : 1.f);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __half2 y = __floats2half2_rn(bf_lo(x[s][i]) * down, bf_hi(x[s][i]) * down);
          x[s][i] = *reinterpret_cast<const uint32_t*>(&y);
        }
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      qa[s][r] = x[s][0];
      qa[s][(kWide ? 2 : 1) + r] = x[s][1];
    }
  }
  __syncthreads();

  // Lane parts of the addresses: 32 lanes copy kRowsPer rows at a time, a chunk each.
  constexpr int kRowsPer = 32 / T::kChunks;
  constexpr int kSwz = T::kChunks >= 8 ? 7 : 3;           // a 64-byte row has four chunks to permute
  const uint64_t policy = passing(), keep = staying();
  const int row_l = lane / T::kChunks, chunk_l = lane % T::kChunks;
  const uint8_t* kb = p.c.k + h * p.c.k_head + row_l * p.c.k_slot + 16 * chunk_l;
  const uint8_t* vb = p.c.v + h * p.c.v_head + row_l * p.c.v_slot + 16 * chunk_l;
  const int page_mask = (1 << p.c.page_shift) - 1;
  const int tiles = (cnt + T::kSlots - 1) / T::kSlots;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(rings)) + warp * T::kRing;

  // Slots in use of each half of a tile (0 for one on a bad page).
  auto limits = [&](int tile, int half) {
    const int at = tile * T::kSlots + 8 * half;             // slot within this CTA's range
    const int lim = min(max(cnt - at, 0), 8);
    return lim > 0 && pages[((lo + at) >> p.c.page_shift) - e0] >= 0 ? lim : 0;
  };
  // Starts the copies of a tile.  A half in use is copied whole (its page holds 8 rows), one that is not stays as it
  // is in the ring.
  auto fetch = [&](int tile, int stage) {
    const uint32_t to = ring + stage * T::kBytes;
#pragma unroll
    for (int half = 0; half < T::kH; ++half) {
      const int at = tile * T::kSlots + 8 * half;
      if (at >= cnt) break;
      const int page = pages[((lo + at) >> p.c.page_shift) - e0];
      if (page < 0) continue;
      const int off = (lo + at) & page_mask;
      const uint8_t* kp = kb + page * p.c.k_page + off * p.c.k_slot;
      const uint8_t* vp = vb + page * p.c.v_page + off * p.c.v_slot;
#pragma unroll
      for (int i = 0; i < (8 + kRowsPer - 1) / kRowsPer; ++i) {
        const int r = 8 * half + i * kRowsPer + row_l;
        const uint32_t dst = to + r * T::kRow + 16 * (chunk_l ^ (swizzle(r) & kSwz));
        copy16(dst, kp + i * kRowsPer * p.c.k_slot, policy);
        copy16(dst + T::kSlots * T::kRow, vp + i * kRowsPer * p.c.v_slot, policy);
      }
    }
  };

  // Running state of head rows g (0) and g + 8 (1, wide): max, this lane's part of the sum, out.
  float m[kWide ? 2 : 1], l[kWide ? 2 : 1];
#pragma unroll
  for (int r = 0; r < (kWide ? 2 : 1); ++r) m[r] = -INFINITY, l[r] = 0.f;
  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  auto compute = [&](int tile, int stage) {
    const uint32_t kt = ring + stage * T::kBytes, vt = kt + T::kSlots * T::kRow;
    int lim[T::kH];
#pragma unroll
    for (int half = 0; half < T::kH; ++half) lim[half] = limits(tile, half);
    float s[T::kH][4];
#pragma unroll
    for (int half = 0; half < T::kH; ++half) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[half][e] = 0.f;
#pragma unroll
      for (int j = 0; j < T::kK; ++j) {
        const uint4 kx = lds16(kt + (8 * half + g) * T::kRow + 16 * ((t + 4 * j) ^ (swizzle(g) & kSwz)));
        const uint32_t w[4] = {kx.x, kx.y, kx.z, kx.w};
        if constexpr (kF8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int st = 4 * j + i;
            mma16<true>(s[half], qa[st][0], kWide ? qa[st][1] : 0u, qa[st][kWide ? 2 : 1], kWide ? qa[st][kWide ? 3 : 0] : 0u,
                        e4m3x2_to_f16x2(w[i] & 0xffffu), e4m3x2_to_f16x2(w[i] >> 16));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int st = 2 * j + i;
            mma16<false>(s[half], qa[st][0], kWide ? qa[st][1] : 0u, qa[st][kWide ? 2 : 1], kWide ? qa[st][kWide ? 3 : 0] : 0u,
                         w[2 * i], w[2 * i + 1]);
          }
        }
      }
    }
    // Scale, mask, and the tile's maximum over the four lanes of a head row.
    float top[kWide ? 2 : 1];
#pragma unroll
    for (int r = 0; r < (kWide ? 2 : 1); ++r) {
      float y = -INFINITY;
#pragma unroll
      for (int half = 0; half < T::kH; ++half)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& z = s[half][2 * r + e];
          z = (2 * t + e < lim[half]) ? z * qs[r] : -INFINITY;
          y = fmaxf(y, z);
        }
      if (p.scores != nullptr && g + 8 * r < G) {
        float* to = p.scores + (bg0 + g + 8 * r) * p.score_pitch + lo + tile * T::kSlots + 2 * t;
#pragma unroll
        for (int half = 0; half < T::kH; ++half)
          store_staying(to + 8 * half, s[half][2 * r], s[half][2 * r + 1], keep);
      }
      y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
      y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
      top[r] = fmaxf(m[r], y);
    }
    bool grown = top[0] > m[0];
    if constexpr (kWide) grown = grown || top[1] > m[1];
    if (__any_sync(0xffffffffu, grown)) {
      float f[kWide ? 2 : 1];
#pragma unroll
      for (int r = 0; r < (kWide ? 2 : 1); ++r) {
        f[r] = m[r] == top[r] ? 1.f : ex2(m[r] - top[r]);   // 0 for a row that had nothing yet
        m[r] = top[r];
        l[r] *= f[r];
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        o[i][0] *= f[0];
        o[i][1] *= f[0];
        o[i][2] *= f[kWide ? 1 : 0];
        o[i][3] *= f[kWide ? 1 : 0];
      }
    }
    // Probabilities, as the A operand of the second product.
    uint32_t hi[T::kH][kWide ? 2 : 1], low[T::kH][kWide ? 2 : 1];
#pragma unroll
    for (int r = 0; r < (kWide ? 2 : 1); ++r) {
      const float base = (m[r] == -INFINITY ? 0.f : m[r]) - kShift;
#pragma unroll
      for (int half = 0; half < T::kH; ++half) {
        const float a = ex2(s[half][2 * r] - base), c = ex2(s[half][2 * r + 1] - base);
        l[r] += a + c;
        split_pair<kF8>(a, c, hi[half][r], low[half][r]);
      }
    }
    auto second = [&](float (&c)[4], int kk, uint32_t b0, uint32_t b1) {
      if constexpr (kWide) {
        mma16<kF8>(c, hi[kk][0], hi[kk][kWide ? 1 : 0], hi[kk + 1][0], hi[kk + 1][kWide ? 1 : 0], b0, b1);
        mma16<kF8>(c, low[kk][0], low[kk][kWide ? 1 : 0], low[kk + 1][0], low[kk + 1][kWide ? 1 : 0], b0, b1);
      } else {
        mma16<kF8>(c, hi[kk][0], low[kk][0], hi[kk + 1][0], low[kk + 1][0], b0, b1);
      }
    };
#pragma unroll
    for (int kk = 0; kk < T::kH; kk += 2)
#pragma unroll
    for (int j = 0; j < T::kV; ++j) {
      // Rows 2t, 2t + 1, 2t + 8, 2t + 9.  Rows past the slots in use hold anything: 0 x NaN must not reach the sums.
      uint32_t w[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int in_half = 2 * t + (r & 1), rr = 8 * (kk + (r >> 1)) + in_half;
        uint4 vx = make_uint4(0, 0, 0, 0);
        if constexpr (T::kRow >= 128) {
          vx = lds16(vt + rr * T::kRow + 16 * ((g + 8 * j) ^ swizzle(in_half)));
        } else {
          const uint2 y = lds8(vt + rr * T::kRow + 16 * ((g >> 1) ^ (swizzle(in_half) & kSwz)) + 8 * (g & 1));
          vx.x = y.x, vx.y = y.y;
        }
        if (in_half >= lim[kk + (r >> 1)]) vx = make_uint4(0, 0, 0, 0);
        w[r][0] = vx.x, w[r][1] = vx.y, w[r][2] = vx.z, w[r][3] = vx.w;
      }
      if constexpr (kF8) {
#pragma unroll
        for (int i = 0; i < (T::kRow >= 128 ? 4 : 2); ++i) {
          const uint32_t x0 = __byte_perm(w[0][i], w[1][i], 0x5140), x1 = __byte_perm(w[2][i], w[3][i], 0x5140);
          const uint32_t y0 = __byte_perm(w[0][i], w[1][i], 0x7362), y1 = __byte_perm(w[2][i], w[3][i], 0x7362);
          second(o[4 * i], kk, e4m3x2_to_f16x2(x0 & 0xffffu), e4m3x2_to_f16x2(x1 & 0xffffu));
          second(o[4 * i + 1], kk, e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(x1 >> 16));
          second(o[4 * i + 2], kk, e4m3x2_to_f16x2(y0 & 0xffffu), e4m3x2_to_f16x2(y1 & 0xffffu));
          second(o[4 * i + 3], kk, e4m3x2_to_f16x2(y0 >> 16), e4m3x2_to_f16x2(y1 >> 16));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          second(o[8 * j + 2 * i], kk, __byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x5410));
          second(o[8 * j + 2 * i + 1], kk, __byte_perm(w[0][i], w[1][i], 0x7632), __byte_perm(w[2][i], w[3][i], 0x7632));
        }
      }
    }
  };

  // kStages - 1 tiles ahead of the one that is computed.
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) {
    if (warp + i * kPdWarps < tiles) fetch(warp + i * kPdWarps, i);
    copy_commit();
  }
  int stage = 0;
  for (int tile = warp; tile < tiles; tile += kPdWarps) {
    copy_wait<T::kStages - 2>();
    __syncwarp();                                         // every lane's copies of this tile, and its reads of the last
    const int ahead = tile + (T::kStages - 1) * kPdWarps;
    if (ahead < tiles) fetch(ahead, stage == 0 ? T::kStages - 1 : stage - 1);
    copy_commit();
    compute(tile, stage);
    stage = stage == T::kStages - 1 ? 0 : stage + 1;
  }
  copy_wait<0>();
  grid_launch_next();
  __syncthreads();                                        // the rings are free

  // Join the warps: every lane holds part of its rows' sums, all four lanes of a row the same maximum.
#pragma unroll
  for (int r = 0; r < (kWide ? 2 : 1); ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (t == 0) {
      sm_m[warp][g + 8 * r] = m[r];
      sm_l[warp][g + 8 * r] = l[r];
    }
  }
  // Column n of out tile i is a head dim that follows from V's chunks: bf16: 64 (i / 8) + 8 n + i % 8;
  // e4m3: (d / 8) n + i.  This lane holds n = 2 t and 2 t + 1.
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = kF8 ? (D / 8) * (2 * t + e) + i : 64 * (i / 8) + 8 * (2 * t + e) + (i % 8);
      if constexpr (kWide) {
        sm_o[warp][g][col] = o[i][e];
        sm_o[warp][g + 8][col] = o[i][2 + e];
      } else {
        sm_o[warp][g][col] = o[i][e] + o[i][2 + e];
      }
    }
  __syncthreads();
  const float vs = kF8 && p.c.v_scale != nullptr ? p.c.v_scale[h] : 1.f;
  // This CTA's maximum, sum and out (a row of D per head), over its warps.
  float (*cta_o)[D] = reinterpret_cast<float (*)[D]>(rings + kPdWarps * kRows * D * sizeof(float));
  static_assert((kPdWarps + 1) * kRows * D * 4 <= kPdWarps * T::kRing, "outputs of the warps and of the CTA");
  __shared__ float2 cta_ml[kRows];
  for (int idx = threadIdx.x; idx < G * D; idx += kPdThreads) {
    const int i = idx / D, d = idx - i * D;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kPdWarps; ++w) top = fmaxf(top, sm_m[w][i]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kPdWarps; ++w) {
      const float f = ex2(sm_m[w][i] - base);
      sum += sm_l[w][i] * f;
      acc += sm_o[w][i][d] * f;
    }
    if (p.cluster) {
      cta_o[i][d] = acc;
      if (d == 0) cta_ml[i] = make_float2(top - kShift, sum);
    } else {
      p.part_o[((bg0 + i) * p.n_split + split) * D + d] = acc * vs;
      if (d == 0) p.part_ml[(bg0 + i) * p.n_split + split] = make_float2(top - kShift, sum);
    }
  }
  if (!p.cluster) return;

  // The cluster's active CTAs see one another's parts through distributed shared memory.
  cg::cluster_group cluster = cg::this_cluster();
  if (active > 1) cluster.sync();
  else __syncthreads();
  __shared__ float2 all_ml[kPdMaxCluster][kRows];         // then .x = the split's share of the row
  __shared__ float lse2[kRows];                           // log2 units; +inf: nothing to add
  for (int idx = threadIdx.x; idx < active * G; idx += kPdThreads) {
    const int q = idx / G, i = idx - q * G;
    all_ml[q][i] = active > 1 ? *cluster.map_shared_rank(&cta_ml[i], q) : cta_ml[i];
  }
  __syncthreads();
  if (threadIdx.x < G) {
    const int i = threadIdx.x;
    float top = -INFINITY, sum = 0.f;
    for (int q = 0; q < active; ++q) top = fmaxf(top, all_ml[q][i].x);
    const float base = top == -INFINITY ? 0.f : top;
    for (int q = 0; q < active; ++q) {
      const float f = ex2(all_ml[q][i].x - base);
      sum += all_ml[q][i].y * f;
      all_ml[q][i].x = f;
    }
    const float inv = sum != 0.f ? vs / sum : 0.f;
    for (int q = 0; q < active; ++q) all_ml[q][i].x *= inv;
    lse2[i] = sum != 0.f ? base + log2f(sum) : INFINITY;
    if (split == 0 && p.lse != nullptr) p.lse[bg0 + i] = sum != 0.f ? lse2[i] * kLn2 : -INFINITY;
  }
  __syncthreads();
  // Each active CTA writes its share of out, two dims per thread.
  for (int idx = split * kPdThreads + threadIdx.x; idx < G * (D / 2); idx += active * kPdThreads) {
    const int i = idx / (D / 2), d = 2 * (idx - i * (D / 2));
    float2 y = make_float2(0.f, 0.f);
    const float2* from = reinterpret_cast<const float2*>(&cta_o[i][d]);
    for (int q0 = 0; q0 < active; q0 += 8) {              // eight peers' values on their way at a time
      float2 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < active) x[q] = active > 1 ? *cluster.map_shared_rank(from, q0 + q) : *from;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < active) {
          const float f = all_ml[q0 + q][i].x;
          if (f != 0.f) y.x += x[q].x * f, y.y += x[q].y * f;
        }
    }
    const __nv_bfloat162 z = __floats2bfloat162_rn(y.x, y.y);
    *reinterpret_cast<uint32_t*>(p.out + (bg0 + i) * D + d) = *reinterpret_cast<const uint32_t*>(&z);
  }
  // weight[c] += sum over the group of 2^(s - lse2): this CTA's own scores, four slots (of one page) per thread.
  if (p.scores != nullptr) {
    for (int at = 4 * threadIdx.x; at < cnt; at += 4 * kPdThreads) {
      const int page = pages[((lo + at) >> p.c.page_shift) - e0];
      float add[4] = {0.f, 0.f, 0.f, 0.f};
      const float* from = p.scores + bg0 * p.score_pitch + lo + at;
      float* to = p.c.weight + ((static_cast<int64_t>(max(page, 0)) * p.c.n_kv_heads + h) << p.c.page_shift) + ((lo + at) & page_mask);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (page >= 0) w = *reinterpret_cast<const float4*>(to);
#pragma unroll
      for (int i0 = 0; i0 < kRows; i0 += 8) {
        float4 s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i < G) s[i] = *reinterpret_cast<const float4*>(from + (i0 + i) * static_cast<int64_t>(p.score_pitch));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i < G) {
            const float z = lse2[i0 + i];
            add[0] += ex2(s[i].x - z), add[1] += ex2(s[i].y - z), add[2] += ex2(s[i].z - z), add[3] += ex2(s[i].w - z);
          }
      }
      if (page < 0) continue;
      if (at + 3 < cnt) {
        *reinterpret_cast<float4*>(to) = make_float4(w.x + add[0], w.y + add[1], w.z + add[2], w.w + add[3]);
      } else {
        const float old[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (at + e < cnt) to[e] = old[e] + add[e];
      }
    }
  }
  if (active > 1) cluster.sync();                         // the peers have read this CTA's parts
}

// Joins the splits of a row and adds the probabilities to the weights.  CTA
// (x, y): row x, slots y, y + gridDim.y, ... of kPjSlots each, and of the
// group's heads those with index y modulo gridDim.y.  With lse2 of every head
// known (a warp each), the parts and scores need one factor:
//   out = sum over splits of part 2^(max - lse2),  weight[c] += sum over heads of 2^(score - lse2)
// Scores were written moments ago and are mostly still in the L2; what costs
// is the chain of loads and the few instructions per byte, so a CTA goes
// through a whole row where there are many rows (64 x 8 rows of 4,032 slots:
// JOIN_MEASURED).
constexpr int kPjThreads = 256;
constexpr int kPjWarps = kPjThreads / 32;
constexpr int kPjSlots = 4 * kPjThreads;
constexpr int kPjMaxGroup = 1024;
constexpr int kPjHeads = 4;                                // heads whose scores are asked for together

template <int D>
__global__ void __launch_bounds__(kPjThreads, 4) paged_join_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr int kWords = D / 4;                            // 16-byte words of a part's row
  constexpr int kParts = kPjThreads / kWords;              // splits read side by side when there are many
  __shared__ float lse2[kPjMaxGroup];                      // log2 units; +inf: nothing to add
  __shared__ float4 acc_s[kParts][kWords];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int64_t bg0 = static_cast<int64_t>(b) * p.n_q_heads + static_cast<int64_t>(h) * p.group;
  const int ns = p.n_split;
  grid_wait();
  grid_launch_next();
  const int count = p.c.count[row];
  // A step's pages and scores do not depend on anything: the first step's are on their way from here on.
  const float* scores = p.scores + bg0 * p.score_pitch;
  const int32_t* table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
  int at = blockIdx.y * kPjSlots + 4 * tid;
  int page = -1;
  float4 s[kPjHeads];
  auto ask = [&](int slot, int g0) {
#pragma unroll
    for (int i = 0; i < kPjHeads; ++i)
      if (slot < p.c.capacity && g0 + i < p.group)
        s[i] = __ldcg(reinterpret_cast<const float4*>(scores + (g0 + i) * static_cast<int64_t>(p.score_pitch) + slot));
  };
  if (p.scores != nullptr) {
    if (at < p.c.capacity) page = table[at >> p.c.page_shift];
    ask(at, 0);
  }
  for (int i = warp; i < p.group; i += kPjWarps) {
    const float2* ml = p.part_ml + (bg0 + i) * ns;
    float top = -INFINITY, sum = 0.f;
    for (int j = lane; j < ns; j += 32) {
      const float2 x = ml[j];
      const float up = fmaxf(top, x.x), base = up == -INFINITY ? 0.f : up;
      sum = sum * ex2(top - base) + x.y * ex2(x.x - base);
      top = up;
    }
    float all = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    all = all == -INFINITY ? 0.f : all;
    sum *= ex2(top - all);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      lse2[i] = sum != 0.f ? all + log2f(sum) : INFINITY;
      if (blockIdx.y == 0 && p.lse != nullptr) p.lse[bg0 + i] = sum != 0.f ? (all + log2f(sum)) * kLn2 : -INFINITY;
    }
  }
  __syncthreads();
  const int n = min(max(count, 0), p.c.capacity);

  // out: splits without slots wrote no part (max -inf, sum 0).
  auto add_split = [&](float4& acc, int64_t bg, int j, int w, float z) {
    const float2 x = p.part_ml[bg * ns + j];
    if (x.x == -INFINITY && x.y == 0.f) return;
    const float f = ex2(x.x - z);
    const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + (bg * ns + j) * D + 4 * w));
    acc.x += y.x * f, acc.y += y.y * f, acc.z += y.z * f, acc.w += y.w * f;
  };
  auto write_out = [&](int64_t bg, int w, const float4& y, float z) {
    const bool some = z != INFINITY;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(some ? y.x : 0.f, some ? y.y : 0.f);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(some ? y.z : 0.f, some ? y.w : 0.f);
    *reinterpret_cast<uint2*>(p.out + bg * D + 4 * w) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  };
  if (ns <= kParts) {
    // A thread per word.
    const int heads = (p.group - static_cast<int>(blockIdx.y) + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
    for (int idx = tid; idx < heads * kWords; idx += kPjThreads) {
      const int i = blockIdx.y + idx / kWords * gridDim.y, w = idx % kWords;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int j = 0; j < ns; ++j) add_split(acc, bg0 + i, j, w, lse2[i]);
      write_out(bg0 + i, w, acc, lse2[i]);
    }
  } else {
    // kParts threads per word, each with every kParts-th split.
    for (int i = blockIdx.y; i < p.group; i += gridDim.y) {
      const int w = tid % kWords, part = tid / kWords;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int j = part; j < ns; j += kParts) add_split(acc, bg0 + i, j, w, lse2[i]);
      acc_s[part][w] = acc;
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int q = 1; q < kParts; ++q) {
          const float4 y = acc_s[q][w];
          acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
        }
        write_out(bg0 + i, w, acc, lse2[i]);
      }
      __syncthreads();
    }
  }
  if (p.scores == nullptr) return;

  // weights: four slots (of one page) per thread and step.
  const int page_mask = (1 << p.c.page_shift) - 1;
  while (at < n) {
    const bool good = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.c.n_pages);     // the attention reports it
    float* to = p.c.weight + ((static_cast<int64_t>(good ? page : 0) * p.c.n_kv_heads + h) << p.c.page_shift) + (at & page_mask);
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (good) w = *reinterpret_cast<const float4*>(to);
    const int next = at + gridDim.y * kPjSlots;
    if (next < n) page = table[next >> p.c.page_shift];
    float add[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g0 = 0; g0 < p.group; g0 += kPjHeads) {
      float4 x[kPjHeads];
#pragma unroll
      for (int i = 0; i < kPjHeads; ++i) x[i] = s[i];
      if (g0 + kPjHeads < p.group) ask(at, g0 + kPjHeads);
      else ask(next, 0);
#pragma unroll
      for (int i = 0; i < kPjHeads; ++i)
        if (g0 + i < p.group) {
          const float z = lse2[g0 + i];
          add[0] += ex2(x[i].x - z), add[1] += ex2(x[i].y - z), add[2] += ex2(x[i].z - z), add[3] += ex2(x[i].w - z);
        }
    }
    if (good) {
      if (at + 3 < n) {
        *reinterpret_cast<float4*>(to) = make_float4(w.x + add[0], w.y + add[1], w.z + add[2], w.w + add[3]);
      } else {
        const float old[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (at + e < n) to[e] = old[e] + add[e];
      }
    }
    at = next;
  }
}

// Slots per CTA: enough CTAs for several rounds of two per SM, so that rows
// of different length even out, and pieces of 128 to 2,048 slots; a second
// kernel joins them.  Where clusters of up to 16 CTAs hold whole rows and all
// fit at once, a row's pieces are a cluster and join in distributed shared
// memory: one launch, and no parts in the workspace.  CLUSTER_MEASURED
DecodeSplit paged_split(int64_t rows, int capacity, bool may_cluster) {
  constexpr int64_t kWave = 148 * 2;
  if (may_cluster) {
    int n = 1;
    while (n < kPdMaxCluster && n * 128 < capacity) n *= 2;
    const int slots = ((capacity + n - 1) / n + 63) / 64 * 64;
    if (rows * n <= kWave && slots <= kPdMaxSplit) return {slots, n, true};
  }
  int64_t slots = (rows * capacity + 5 * kWave - 1) / (5 * kWave);
  slots = std::max<int64_t>(128, std::min<int64_t>(kPdMaxSplit, (slots + 63) / 64 * 64));
  return {static_cast<int>(slots), static_cast<int>((capacity + slots - 1) / slots), false};
}

template <int D, bool kF8>
static cudaError_t launch_decode_of(const PagedDecodeParams& p, int64_t rows, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.cluster ? rows * p.n_split : rows), p.cluster ? 1 : p.n_split), block(kPdThreads);
  constexpr size_t smem = kPdWarps * Tile<D, kF8>::kRing;
  static std::atomic<uint64_t> ready[2];
  auto go = [&](auto kern, int wide) {
    const cudaError_t e = allow_smem(kern, smem, ready[wide], true);
    return e != cudaSuccess ? e : launch_paged(kern, grid, block, smem, p.cluster ? p.n_split : 1, stream, p);
  };
  const cudaError_t e = p.group > 8 ? go(paged_decode_kernel<D, kF8, true>, 1) : go(paged_decode_kernel<D, kF8, false>, 0);
  if (e != cudaSuccess || p.cluster) return e;
  // Join: a CTA per row where that is a wave, else up to one per kPjSlots slots (or per head, without weights).
  const int64_t kv_rows = static_cast<int64_t>(p.c.batch) * p.c.n_kv_heads;
  const int most = p.scores != nullptr ? (p.c.capacity + kPjSlots - 1) / kPjSlots : std::min(p.group, 16);
  const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, 148 * 4 / kv_rows)));
  return launch_paged(paged_join_kernel<D>, dim3(static_cast<unsigned>(kv_rows), parts), dim3(kPjThreads), 0, 1, stream, p);
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int head_dim, bool f8, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.c.batch) * p.c.n_kv_heads * p.head_chunks;
  if (head_dim == 128) return f8 ? launch_decode_of<128, true>(p, rows, stream) : launch_decode_of<128, false>(p, rows, stream);
  return f8 ? launch_decode_of<64, true>(p, rows, stream) : launch_decode_of<64, false>(p, rows, stream);
}

}  // namespace kvpop
