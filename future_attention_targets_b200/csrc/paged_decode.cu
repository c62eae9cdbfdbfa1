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
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kvpop_paged.cuh"

namespace kvpop {

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdChunk = 2048;              // slots whose pages are at hand
constexpr int kPdMinPage = 8;
constexpr float kLn2 = 0.6931471805599453f;

// K and V pass through the L2 once: they are the first to leave it, and the scores written meanwhile the last, so that
// they are still there when the weights are added.  They are read as usual then.  Marked as the first to leave at that
// last use they cost more (96 x 4 e4m3 rows of 8,192 slots 182.3 us against 180.6 among others, 175 against 169 in a
// graph; 64 x 8 rows of 4,032 slots 190.8 against 189.5 among others, though 184 against 185.7 in a graph), and no kernel
// that ran next was faster for it (matrix products, the dense pass 1, an append, passes over 8 to 96 MB).
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
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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

// V's scale of head h (1 without one) as a factor from [1, 2) and a power of two, both exact.  The factor goes with the
// sums, the power with the result: the whole scale over a sum of up to 2^25, or times one, leaves fp32's range long
// before the result does.  Ordinary scales give the same bits either way.
__device__ __forceinline__ float2 split_scale(const float* scales, int h) {
  const float s = scales != nullptr ? scales[h] : 1.f;
  const float up = s < 0x1p-126f ? 0x1p-64f : 1.f;        // subnormal ones by way of 2^64 times them
  const uint32_t u = __float_as_uint(s * (1.f / up));
  return make_float2(__uint_as_float((u & 0x007fffffu) | 0x3f800000u), __uint_as_float(u & 0x7f800000u) * up);
}

// A tile in shared memory: K rows, then V rows.  Rows of 256 bytes come 16 at a
// time, shorter ones 32: a step's chain of products, maximum, exponentials and
// products costs about the same either way, and an e4m3 cache with half the
// bytes per slot was bound by that chain (96 x 4 rows of 8,192 slots: 226 us
// with 16, 206 us with 32).
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
  // Whether a CTA adds the weights of long rows that it does whole, rather than the second kernel (256 x 8 rows of
  // 4,032 slots: 690 us against 720; short rows are left to the second kernel's many warps: 256 x 8 rows of 1 to 4,032
  // slots 107 against 117).  With three CTAs per SM its registers would spill in the attention loop (256 x 8 e4m3
  // rows: 496 against 392).
  static constexpr bool kSums = kRow == 256;
  static constexpr int kRing = kStages * kBytes;                // bytes of a warp's ring
};

// Chunk permutation of row r within a tile.
__device__ __forceinline__ int swizzle(int r) { return (r & 6) ^ ((r & 1) << 2); }

// How the rows are dealt out.  An item is a row (b, h) and up to 16 of its
// query heads.  It counts as its blocks of 128 slots in use, and kPdItem more
// for what starting and ending an item costs; the items in line are cut into
// equal shares, one per CTA, as many CTAs as the SMs hold.  So whatever the
// rows' lengths, every CTA has the same to do and none starts for an empty row.
// A share covers the end of one item, whole items and the start of another;
// an item in several shares leaves parts (maximum, sum, out) for the second
// kernel: the one that starts it in its CTA's place 1, the others in place 0.
// Every CTA finds its share from the counts.
constexpr int kPdBlock = 128;
constexpr int kPdItem = 2;
constexpr int kPdSumSlots = 1024;           // a whole row's weights are added by its CTA from this many slots on
constexpr int kPdItemsHeld = 1024;          // items whose sizes a CTA keeps at hand

__device__ __forceinline__ int item_slots(const PagedDecodeParams& p, int item) {
  return min(max(p.c.count[item / p.head_chunks], 0), p.c.capacity);
}
__device__ __forceinline__ int size_of(int slots) { return slots > 0 ? (slots + kPdBlock - 1) / kPdBlock + kPdItem : 0; }

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
  __shared__ int32_t pages[2][kPdChunk / kPdMinPage + 1];   // of the chunk at work and the next
  __shared__ float sm_m[kPdWarps][kRows], sm_l[kPdWarps][kRows];
  __shared__ int32_t share_s[2];            // first item of this CTA's share, where it begins
  __shared__ int32_t warp_sizes[kPdWarps];
  __shared__ int32_t slots_held[kPdItemsHeld];
  __shared__ int32_t bad_pages;             // the segment has pages that the pool does not
  __shared__ float2 fin[kRows];             // factor of out (1 / sum), lse2 (+inf: nothing to add)
  extern __shared__ __align__(128) uint8_t rings[];
  float (*sm_o)[kRows][D] = reinterpret_cast<float (*)[kRows][D]>(rings);   // once the rings are done with
  static_assert(kRows * D * 4 <= T::kRing, "the warps' outputs reuse their rings");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int items = p.c.batch * p.c.n_kv_heads * p.head_chunks;
  const uint64_t policy = passing(), keep = staying();
  if (threadIdx.x == 0) bad_pages = 0;
  __syncthreads();
  grid_wait();
  grid_launch_next();                       // the next kernel's CTAs come in as these leave, and wait for the last

  const bool held = items <= kPdItemsHeld && !p.whole;
  auto slots_of = [&](int i) { return held ? slots_held[i] : item_slots(p, i); };
  int item = blockIdx.x;
  int x = 0, x1 = 1, before = 0;            // this CTA's share of the line; where the item begins
  if (!p.whole) {
    // Where each thread's run of items begins, by a scan over the threads' sums.
    const int per = (items + kPdThreads - 1) / kPdThreads;
    const int i0 = min(items, static_cast<int>(threadIdx.x) * per), i1 = min(items, i0 + per);
    int mine = 0;
#pragma unroll 8
    for (int i = i0; i < i1; ++i) {
      const int slots = item_slots(p, i);
      mine += size_of(slots);
      if (held) slots_held[i] = slots;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sizes[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kPdWarps; ++w) {
      if (w < warp) incl += warp_sizes[w];
      total += warp_sizes[w];
    }
    const int share = max(1, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
    x = min(total, static_cast<int>(blockIdx.x) * share);   // no overflow: total + CTAs is below 2^31
    x1 = min(total, x + share);
    const int start = incl - mine;
    if (start <= x && x < incl) {           // one thread's run holds the share's beginning
      int at = start, i = i0;
      for (int size = size_of(slots_of(i)); at + size <= x; size = size_of(slots_of(i))) at += size, ++i;
      share_s[0] = i;
      share_s[1] = at;
    }
    if (blockIdx.x == 0) {                  // for the second kernel: the CTA of each item's first slots, and how many
      int at = start;
      for (int i = i0; i < i1; ++i) {
        const int size = size_of(slots_of(i));
        const int c0 = (at + kPdItem) / share;
        p.item_parts[i] = make_int2(c0, size > 0 ? (at + size - 1) / share - c0 + 1 : 0);
        at += size;
      }
    }
    __syncthreads();
    if (x >= x1) return;
    item = share_s[0];
    before = share_s[1];
  }

  for (; x < x1; ++item) {
  const int hc = item % p.head_chunks;                    // chunk of 16 heads of the group
  const int row = item / p.head_chunks;                   // (b, h)
  const int b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int G = min(p.group - hc * 16, 16);               // query heads of this item
  const int64_t bg0 = static_cast<int64_t>(b) * p.n_q_heads + h * p.group + hc * 16;
  const int n = slots_of(item);
  int lo = 0, cnt = n;                                    // slots of this segment
  if (!p.whole) {
    if (n == 0) continue;
    const int from = x - before - kPdItem, to = x1 - before - kPdItem;    // in blocks of the item
    lo = max(0, from) * kPdBlock;
    cnt = min(static_cast<int64_t>(n), static_cast<int64_t>(max(0, to)) * kPdBlock) - lo;
    before += size_of(n);
    x = before;
    if (cnt <= 0) continue;                               // the share ends before the item's first slots
  } else {
    x = 1;
    if (n == 0) {
      for (int i = threadIdx.x; i < G * D; i += kPdThreads) p.out[bg0 * D + i] = 0;
      if (p.lse != nullptr)
        for (int i = threadIdx.x; i < G; i += kPdThreads) p.lse[bg0 + i] = -INFINITY;
      continue;
    }
  }
  // The pages of a chunk of slots; one that the pool does not have is -1 from here on.
  const int shift = p.c.page_shift;
  auto entry0 = [&](int chunk) { return (lo + chunk * kPdChunk) >> shift; };
  auto stage_pages = [&](int chunk) {
    const int e0 = entry0(chunk), e1 = (lo + min(cnt, (chunk + 1) * kPdChunk) - 1) >> shift;
    for (int i = threadIdx.x; i <= e1 - e0; i += kPdThreads) {
      const int page = page_of(p.c, b, e0 + i, p.status, DBG_PAGED_DECODE, 1);
      pages[chunk & 1][i] = page;
      if (page < 0) bad_pages = 1;
    }
  };
  const int chunks = (cnt + kPdChunk - 1) / kPdChunk;

  // q in the order of K's chunks: A operand rows g and (wide) g + 8.  Its loads and the pages' go out together.
  uint32_t qa[KS][kWide ? 4 : 2];
  float qs[kWide ? 2 : 1];                                // score per unit of product, log2 units
  uint4 qw[kWide ? 2 : 1][D / 32];
#pragma unroll
  for (int r = 0; r < (kWide ? 2 : 1); ++r)
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      // bf16 cache: chunk j holds dims 32 j + 8 t + 0..7, two k steps; e4m3: dims 64 j' + 16 t + 0..15, four.
      const int d0 = kF8 ? 64 * (j / 2) + 16 * t + 8 * (j & 1) : 32 * j + 8 * t, head = g + 8 * r;
      qw[r][j] = make_uint4(0, 0, 0, 0);
      if (head < G)
        qw[r][j] = *reinterpret_cast<const uint4*>(p.q + b * p.q_stride + static_cast<int64_t>(h * p.group + hc * 16 + head) * D + d0);
    }
  stage_pages(0);
#pragma unroll
  for (int r = 0; r < (kWide ? 2 : 1); ++r) {
    uint32_t x[KS][2];                                    // bf16 pairs: k step s, first and second half
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      x[2 * j][0] = qw[r][j].x, x[2 * j][1] = qw[r][j].y, x[2 * j + 1][0] = qw[r][j].z, x[2 * j + 1][1] = qw[r][j].w;
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
  // Lane parts of the addresses: 32 lanes copy kRowsPer rows at a time, a chunk each.
  constexpr int kRowsPer = 32 / T::kChunks;
  constexpr int kSwz = T::kChunks >= 8 ? 7 : 3;           // a 64-byte row has four chunks to permute
  const int row_l = lane / T::kChunks, chunk_l = lane % T::kChunks;
  const uint32_t k_page = static_cast<uint32_t>(p.c.k_page), v_page = static_cast<uint32_t>(p.c.v_page);   // below 4 GiB
  const uint32_t k_slot = static_cast<uint32_t>(p.c.k_slot), v_slot = static_cast<uint32_t>(p.c.v_slot);
  const uint8_t* kb = p.c.k + h * p.c.k_head + static_cast<uint64_t>(k_slot) * row_l + 16 * chunk_l;
  const uint8_t* vb = p.c.v + h * p.c.v_head + static_cast<uint64_t>(v_slot) * row_l + 16 * chunk_l;
  const int page_mask = (1 << shift) - 1;
  const int tiles = (cnt + T::kSlots - 1) / T::kSlots;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(rings)) + warp * T::kRing;

  // Page of slot lo + at.
  auto page_at = [&](int at) {
    const int chunk = at / kPdChunk;
    if (!KVPOP_IN(at >= 0 && at < cnt && ((lo + at) >> shift) - entry0(chunk) <= kPdChunk / kPdMinPage, p.dbg, DBG_PAGED_DECODE, 2))
      return -1;
    return pages[chunk & 1][((lo + at) >> shift) - entry0(chunk)];
  };
  // Starts the copies of rows kFirst .. kFirst + kN - 1 of a tile, which lie on one page from slot lo + at on.  They
  // are copied whole: a page holds them all, in use or not.
  auto fetch_rows = [&](uint32_t to, int at, auto first, auto count) {
    constexpr int kFirst = decltype(first)::value, kN = decltype(count)::value;
    const int page = page_at(at);
    if (page < 0) return;                                 // stays as it is in the ring
    const int off = (lo + at) & page_mask;
    KVPOP_CHECK(off + kN <= page_mask + 1, p.dbg, DBG_PAGED_DECODE, 3);
    const uint8_t* kp = kb + static_cast<uint64_t>(static_cast<uint32_t>(page)) * k_page + static_cast<uint64_t>(off) * k_slot;
    const uint8_t* vp = vb + static_cast<uint64_t>(static_cast<uint32_t>(page)) * v_page + static_cast<uint64_t>(off) * v_slot;
#pragma unroll
    for (int i = 0; i < (kN + kRowsPer - 1) / kRowsPer; ++i) {
      const int r = kFirst + i * kRowsPer + row_l;
      const uint32_t dst = to + r * T::kRow + 16 * (chunk_l ^ (swizzle(r) & kSwz));
      copy16(dst, kp + static_cast<uint64_t>(k_slot) * (i * kRowsPer), policy);
      copy16(dst + T::kSlots * T::kRow, vp + static_cast<uint64_t>(v_slot) * (i * kRowsPer), policy);
    }
  };
  auto fetch = [&](int tile, int stage) {
    const uint32_t to = ring + stage * T::kBytes;
    const int at = tile * T::kSlots;
    if ((1 << shift) >= T::kSlots) {                      // segments start at blocks, so a tile is on one page
      fetch_rows(to, at, std::integral_constant<int, 0>(), std::integral_constant<int, T::kSlots>());
    } else {
      fetch_rows(to, at, std::integral_constant<int, 0>(), std::integral_constant<int, 8>());
      if (at + 8 < cnt) fetch_rows(to, at + 8, std::integral_constant<int, 8>(), std::integral_constant<int, 8>());
      if constexpr (T::kSlots == 32) {
        if (at + 16 < cnt) fetch_rows(to, at + 16, std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
        if (at + 24 < cnt) fetch_rows(to, at + 24, std::integral_constant<int, 24>(), std::integral_constant<int, 8>());
      }
    }
  };

  bool has_bad = false;
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
    // Scores in log2 units.
#pragma unroll
    for (int half = 0; half < T::kH; ++half)
#pragma unroll
      for (int e = 0; e < (kWide ? 4 : 2); ++e) s[half][e] *= qs[e / 2];
    // A tile with slots that are not in use: they score -inf, and their rows of V, which hold anything, become 0, for
    // 0 x NaN must not reach the sums.
    if ((tile + 1) * T::kSlots > cnt || has_bad) {
#pragma unroll
      for (int half = 0; half < T::kH; ++half) {
        const int at = tile * T::kSlots + 8 * half;
        int lim = min(max(cnt - at, 0), 8);
        if (lim > 0 && page_at(at) < 0) lim = 0;
#pragma unroll
        for (int e = 0; e < (kWide ? 4 : 2); ++e)
          if (2 * t + (e & 1) >= lim) s[half][e] = -INFINITY;
        for (int i = lane; i < (8 - lim) * T::kChunks; i += 32)
          sts16(vt + (8 * half + lim) * T::kRow + 16 * i, make_uint4(0, 0, 0, 0));
      }
      __syncwarp();
    }
    // The tile's maximum over the four lanes of a head row.
    float top[kWide ? 2 : 1];
#pragma unroll
    for (int r = 0; r < (kWide ? 2 : 1); ++r) {
      float y = -INFINITY;
#pragma unroll
      for (int half = 0; half < T::kH; ++half) y = fmaxf(y, fmaxf(s[half][2 * r], s[half][2 * r + 1]));
      if (p.scores != nullptr && g + 8 * r < G &&
          KVPOP_IN(lo + (tile + 1) * T::kSlots <= p.score_pitch, p.dbg, DBG_PAGED_DECODE, 4)) {
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
      // Rows 2t, 2t + 1, 2t + 8, 2t + 9.
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

  // kStages - 1 tiles ahead of the one that is computed.  The ring runs on from chunk to chunk; the barriers let the
  // next chunk's pages in.
  constexpr int kChunkTiles = kPdChunk / T::kSlots;
  static_assert(kChunkTiles % kPdWarps == 0, "a chunk is the same number of steps for every warp");
  int stage = 0;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    if (chunk > 0) __syncthreads();                       // the chunk before is done with its pages
    if (chunk + 1 < chunks) stage_pages(chunk + 1);
    __syncthreads();
    has_bad = bad_pages != 0;
    if (chunk == 0) {
#pragma unroll
      for (int i = 0; i < T::kStages - 1; ++i) {
        if (warp + i * kPdWarps < tiles) fetch(warp + i * kPdWarps, i);
        copy_commit();
      }
    }
    const int end = min(tiles, (chunk + 1) * kChunkTiles);
    for (int tile = chunk * kChunkTiles + warp; tile < end; tile += kPdWarps) {
      copy_wait<T::kStages - 2>();
      __syncwarp();                                       // every lane's copies of this tile, and its reads of the last
      const int ahead = tile + (T::kStages - 1) * kPdWarps;
      if (ahead < tiles) fetch(ahead, stage == 0 ? T::kStages - 1 : stage - 1);
      copy_commit();
      compute(tile, stage);
      stage = stage == T::kStages - 1 ? 0 : stage + 1;
    }
  }
  copy_wait<0>();
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
  const float2 vs = kF8 ? split_scale(p.c.v_scale, h) : make_float2(1.f, 1.f);
  const bool all = cnt == n;                              // the whole item: the result; else a part of it
  const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (lo == 0 ? 1 : 0)) * 16;
  KVPOP_CHECK(lo + cnt <= n && n <= p.c.capacity && row < p.c.batch * p.c.n_kv_heads, p.dbg, DBG_PAGED_DECODE, 5);
  if (threadIdx.x < G) {
    const int i = threadIdx.x;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kPdWarps; ++w) top = fmaxf(top, sm_m[w][i]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kPdWarps; ++w) {
      const float f = ex2(sm_m[w][i] - base);
      sum += sm_l[w][i] * f;
      sm_m[w][i] = f;                                     // the warp's factor
    }
    const float l2 = sum != 0.f ? base - kShift + log2f(sum) : INFINITY;
    fin[i] = make_float2(all ? (sum != 0.f ? vs.x / sum : 0.f) : vs.x, l2);
    if (all) {
      if (p.lse != nullptr) p.lse[bg0 + i] = sum != 0.f ? l2 * kLn2 : -INFINITY;
      if (!p.whole && p.scores != nullptr) p.row_lse2[bg0 + i] = l2;
    } else {
      p.part_ml[part + i] = make_float2(top - kShift, sum);
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < G * (D / 4); idx += kPdThreads) {
    const int i = idx / (D / 4), d = 4 * (idx - i * (D / 4));
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPdWarps; ++w) {
      const float f = sm_m[w][i];
      const float4 z = *reinterpret_cast<const float4*>(&sm_o[w][i][d]);
      y.x += z.x * f, y.y += z.y * f, y.z += z.z * f, y.w += z.w * f;
    }
    const float f = fin[i].x;
    if (all) {
      const bool some = fin[i].y != INFINITY;
      const __nv_bfloat162 u = __floats2bfloat162_rn(some ? y.x * f * vs.y : 0.f, some ? y.y * f * vs.y : 0.f);
      const __nv_bfloat162 w = __floats2bfloat162_rn(some ? y.z * f * vs.y : 0.f, some ? y.w * f * vs.y : 0.f);
      *reinterpret_cast<uint2*>(p.out + (bg0 + i) * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&w));
    } else {
      *reinterpret_cast<float4*>(p.part_o + (part + i) * D + d) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
    }
  }
  if (all && p.scores != nullptr && p.head_chunks == 1 && (p.whole || (T::kSums && n >= kPdSumSlots))) {
    constexpr int kU = T::kSums ? 2 : 1;
    const int32_t* table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    for (int at0 = 4 * threadIdx.x; at0 < n; at0 += 4 * kU * kPdThreads) {
      float4 w[kU];
      float add[kU][4] = {};
      float* to[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int at = at0 + u * 4 * kPdThreads;
        const int page = at < n ? table[at >> shift] : -1;
        const bool good = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.c.n_pages);
        to[u] = good ? p.c.weight + ((static_cast<int64_t>(page) * p.c.n_kv_heads + h) << shift) + (at & page_mask) : nullptr;
      }
#pragma unroll
      for (int i0 = 0; i0 < kRows; i0 += 8) {
        float4 s[kU][8];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i0 + i < G && at0 + u * 4 * kPdThreads < n)
              s[u][i] = __ldcg(reinterpret_cast<const float4*>(p.scores + (bg0 + i0 + i) * p.score_pitch + at0 + u * 4 * kPdThreads));
        if (i0 == 0)
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (to[u] != nullptr) w[u] = *reinterpret_cast<const float4*>(to[u]);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i0 + i < G) {
              const float z = fin[i0 + i].y;
              add[u][0] += ex2(s[u][i].x - z), add[u][1] += ex2(s[u][i].y - z);
              add[u][2] += ex2(s[u][i].z - z), add[u][3] += ex2(s[u][i].w - z);
            }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (to[u] == nullptr) continue;
        const int at = at0 + u * 4 * kPdThreads;
        if (at + 3 < n) {
          *reinterpret_cast<float4*>(to[u]) =
              make_float4(w[u].x + add[u][0], w[u].y + add[u][1], w[u].z + add[u][2], w[u].w + add[u][3]);
        } else {
          const float old[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (at + e < n) to[u][e] = old[e] + add[u][e];
        }
      }
    }
  }
  __syncthreads();                                        // bad_pages is set no more
  if (threadIdx.x == 0) bad_pages = 0;
  __syncthreads();                                        // before the next item's pages, rings and factors
  }
}

// Joins the splits of a row and adds the probabilities to the weights.  CTA
// (x, y): row x, slots y, y + gridDim.y, ... of kPjSlots each, and of the
// group's heads those with index y modulo gridDim.y.  With lse2 of every head
// known (a warp each), the parts and scores need one factor:
//   out = sum over splits of part 2^(max - lse2),  weight[c] += sum over heads of 2^(score - lse2)
// A cluster of 2 to 16 CTAs per row that joins in distributed shared memory
// instead was slower for 64 x 8 rows of 4,032 slots (203 us in all, 190 with
// this kernel): its end has no loads in flight, and large clusters wait for
// room.  For a few rows, where this kernel is a quarter of the time, it has not
// been tried.
// Scores were written moments ago and are mostly still in the L2; what costs
// is the chain of loads and the few instructions per byte, so a CTA goes
// through many slots of a row (64 x 8 rows of 4,032 slots: 12.8 us, 18.6 with a
// CTA per 512 slots and one per head).
constexpr int kPjThreads = 256;
constexpr int kPjWarps = kPjThreads / 32;
constexpr int kPjSlots = 4 * kPjThreads;
constexpr int kPjMaxGroup = 1024;
constexpr int kPjHeads = 4;                                // heads whose scores are asked for together

template <int D, bool kF8>
__global__ void __launch_bounds__(kPjThreads, 4) paged_join_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr bool kSums = Tile<D, kF8>::kSums;
  constexpr int kWords = D / 4;                            // 16-byte words of a part's row
  constexpr int kParts = kPjThreads / kWords;              // splits read side by side when there are many
  __shared__ float lse2[kPjMaxGroup];                      // log2 units; +inf: nothing to add
  __shared__ float4 acc_s[kParts][kWords];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int64_t bg0 = static_cast<int64_t>(b) * p.n_q_heads + static_cast<int64_t>(h) * p.group;
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
  // A row that one CTA did whole is done with, but for its weights if that does not add them.
  const bool one = p.head_chunks == 1 && p.item_parts[row].y == 1;
  if (one && (p.scores == nullptr || (kSums && min(count, p.c.capacity) >= kPdSumSlots))) return;
  const bool done = p.scores == nullptr;
  // Parts of head i's item: of CTAs x .. x + y - 1, the first in place 1.
  auto parts_of = [&](int i) { return p.item_parts[row * p.head_chunks + i / 16]; };
  auto part_at = [&](const int2& q, int i, int j) {
    KVPOP_CHECK(q.x >= 0 && j < q.y && q.x + j < p.ctas, p.dbg, DBG_PAGED_JOIN, 1);
    return (static_cast<int64_t>(q.x + j) * 2 + (j == 0 ? 1 : 0)) * 16 + i % 16;
  };
  for (int i = warp; i < p.group; i += kPjWarps) {
    const int2 q = parts_of(i);
    float l2 = INFINITY;
    if (q.y == 1) {
      if (p.scores != nullptr) l2 = p.row_lse2[bg0 + i];   // several items: the weights are still to do
    } else {
      float top = -INFINITY, sum = 0.f;
      for (int j = lane; j < q.y; j += 32) {
        const float2 x = p.part_ml[part_at(q, i, j)];
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
      if (sum != 0.f) l2 = all + log2f(sum);
      if (lane == 0 && blockIdx.y == 0 && p.lse != nullptr) p.lse[bg0 + i] = sum != 0.f ? l2 * kLn2 : -INFINITY;
    }
    if (lane == 0) lse2[i] = l2;
  }
  __syncthreads();
  const int n = min(max(count, 0), p.c.capacity);

  // out of this CTA's heads, kParts threads per word, each with every kParts-th part.
  for (int i = blockIdx.y; i < p.group; i += gridDim.y) {
    const int2 q = parts_of(i);
    if (q.y == 1) continue;                            // the attention wrote it
    const int w = tid % kWords, part = tid / kWords;
    const float z = lse2[i];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float up = kF8 ? split_scale(p.c.v_scale, h).y : 1.f;        // the parts have the rest of the scale
    if (z != INFINITY) {
#pragma unroll 4
      for (int j = part; j < q.y; j += kParts) {
        const int64_t from = part_at(q, i, j);
        const float f = ex2(p.part_ml[from].x - z);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + from * D + 4 * w));
        acc.x += y.x * f, acc.y += y.y * f, acc.z += y.z * f, acc.w += y.w * f;
      }
    }
    acc_s[part][w] = acc;
    __syncthreads();
    if (part == 0) {
      for (int o = 1; o < min(kParts, q.y); ++o) {
        const float4 y = acc_s[o][w];
        acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
      }
      const __nv_bfloat162 u = __floats2bfloat162_rn(acc.x * up, acc.y * up), v = __floats2bfloat162_rn(acc.z * up, acc.w * up);
      *reinterpret_cast<uint2*>(p.out + (bg0 + i) * D + 4 * w) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
    }
    __syncthreads();
  }
  if (done) return;

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

// Whole items, one CTA each and no second kernel, where rows are short: up to
// 512 slots (1 x 8 rows of 512: 9.2 us against 10.8 in shares; 64 x 8: 29 and
// 33), up to 1,024 if there are many (16 x 8 rows of 1,000: 16.4 and 22.8, but
// 1 x 8: 14.9 and 11.4).  Longer rows of different lengths would leave the SMs
// to the longest one.  Else as many shares as CTAs fit on 148 SMs (with two
// to four times as many: bf16 1 to 2% faster at 64 x 8 rows of 4,032 slots, 8
// x 8 rows 10 to 30% slower); 0 CTAs: too many.
DecodeSplit paged_split(int64_t items, int capacity, int head_dim, bool f8, bool wide, bool may_be_whole) {
  if (may_be_whole && (capacity <= 512 || (capacity <= 1024 && items >= 64))) return {static_cast<int>(items), true};
  const int per_sm = head_dim == 128 ? (f8 ? Tile<128, true>::ctas(wide) : Tile<128, false>::ctas(wide))
                                     : (f8 ? Tile<64, true>::ctas(wide) : Tile<64, false>::ctas(wide));
  const int64_t sizes = items * ((capacity + kPdBlock - 1) / kPdBlock + kPdItem);
  if (sizes + 148 * per_sm >= (int64_t(1) << 31)) return {0, false};    // the line's places are 32-bit
  return {static_cast<int>(std::min<int64_t>(sizes, 148 * per_sm)), false};
}

template <int D, bool kF8>
static cudaError_t launch_decode_of(const PagedDecodeParams& p, cudaStream_t stream) {
  const dim3 grid(p.ctas), block(kPdThreads);
  constexpr size_t smem = kPdWarps * Tile<D, kF8>::kRing;
  static SmemReady ready[2];
  auto go = [&](auto kern, int wide) {
    const cudaError_t e = allow_smem(kern, smem, ready[wide]);
    return e != cudaSuccess ? e : launch_paged(kern, grid, block, smem, 1, stream, p);
  };
  const cudaError_t e = p.group > 8 ? go(paged_decode_kernel<D, kF8, true>, 1) : go(paged_decode_kernel<D, kF8, false>, 0);
  if (e != cudaSuccess || p.whole) return e;
  // Join: six CTAs per SM or more where rows are few, up to one per kPjSlots slots (or per head, without weights).
  const int64_t rows = static_cast<int64_t>(p.c.batch) * p.c.n_kv_heads;
  const int most = p.scores != nullptr ? (p.c.capacity + kPjSlots - 1) / kPjSlots : std::min(p.group, 16);
  const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (148 * 6 + rows - 1) / rows)));
  return launch_paged(paged_join_kernel<D, kF8>, dim3(static_cast<unsigned>(rows), parts), dim3(kPjThreads), 0, 1, stream, p);
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int head_dim, bool f8, cudaStream_t stream) {
  if (head_dim == 128) return f8 ? launch_decode_of<128, true>(p, stream) : launch_decode_of<128, false>(p, stream);
  return f8 ? launch_decode_of<64, true>(p, stream) : launch_decode_of<64, false>(p, stream);
}

}  // namespace kvpop
