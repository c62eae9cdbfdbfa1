// Compaction of a packed prompt's kept K/V rows into pages, sm_100a.
//
// The slot of a kept position is the number of kept positions before it in
// its sequence.  A CTA takes `block` consecutive positions of one (sequence,
// KV head): it counts the mask bytes before them (16-byte loads from L2; the
// mask is 1/512 of the rows' bytes, so counting it again in every CTA costs
// less than a pass of its own that would hand the counts on), ranks its own
// kept positions by a block scan, and copies their rows.  The kernel is bound
// by the copy's HBM traffic.
#include <algorithm>

#include "kvpop_paged.cuh"

namespace kvpop {

constexpr int kPcThreads = 256;
constexpr int kPcWarps = kPcThreads / 32;
constexpr int kPcMaxBlock = 1024;

__device__ __forceinline__ int block_sum_scan(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPcWarps; ++w) {
    before += w < warp ? sums[w] : 0;
    all += sums[w];
  }
  *total = all;
  return before + incl - x;
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kPcThreads, kF8 ? 5 : 4) paged_compact_kernel(const __grid_constant__ PagedCompactParams p) {
  __shared__ int sums[kPcWarps];
  __shared__ RowEntry list[kPcMaxBlock];
  const int tid = threadIdx.x;
  const int row = blockIdx.x, b = row / p.c.n_kv_heads, h = row - b * p.c.n_kv_heads;
  const int s0 = p.start[b], L = p.start[b + 1] - s0;
  const int p0 = blockIdx.y * p.block;
  if (p0 >= L && blockIdx.y > 0) return;
  const int p1 = min(L, p0 + p.block);
  grid_wait();
  grid_launch_next();
  const uint8_t* mask = p.keep == nullptr ? nullptr : p.keep + static_cast<int64_t>(h) * p.total_tokens + s0;

  // Kept positions before p0.
  int before = p0;
  if (mask != nullptr) {
    int c = 0;
    const int head = min(p0, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(mask) & 15u)) & 15u));
    const int words = (p0 - head) >> 4;
    const uint4* v = reinterpret_cast<const uint4*>(mask + head);
    // Non-zero bytes: bit 7 of ((x & 0x7f) + 0x7f) | x, which cannot carry into the next byte.
    auto bits = [](uint32_t x) { return __popc((((x & 0x7f7f7f7fu) + 0x7f7f7f7fu) | x) & 0x80808080u); };
#pragma unroll 8
    for (int i = tid; i < words; i += kPcThreads) {
      const uint4 x = v[i];
      c += bits(x.x) + bits(x.y) + bits(x.z) + bits(x.w);
    }
    for (int i = tid; i < head; i += kPcThreads) c += mask[i] != 0;
    for (int i = head + 16 * words + tid; i < p0; i += kPcThreads) c += mask[i] != 0;
    block_sum_scan(c, sums, &before);
  }
  // This CTA's kept positions, `per` consecutive ones per thread.
  const int per = p.block / kPcThreads;
  const int first = p0 + tid * per;
  uint32_t kept = 0;
  for (int i = 0; i < per; ++i)
    if (first + i < p1 && (mask == nullptr || mask[first + i] != 0)) kept |= 1u << i;
  int total;
  int rank = block_sum_scan(__popc(kept), sums, &total);
  const int n = min(total, max(0, p.c.capacity - before));
  for (int i = 0; i < per; ++i) {
    if (!((kept >> i) & 1u)) continue;
    if (rank < n && KVPOP_IN(rank >= 0 && rank < kPcMaxBlock && before + rank < p.c.capacity && s0 + first + i < p.total_tokens,
                             p.dbg, DBG_PAGED_COMPACT, 2)) {
      const int slot = before + rank, off = slot & ((1 << p.c.page_shift) - 1);
      const int page = page_of(p.c, b, slot >> p.c.page_shift, p.status, DBG_PAGED_COMPACT, 1);
      list[rank] = row_entry(page, off, first + i);
      if (page >= 0) {
        const int64_t at = ((static_cast<int64_t>(page) * p.c.n_kv_heads + h) << p.c.page_shift) + off;
        if (p.c.pos != nullptr) p.c.pos[at] = first + i;
        if (p.c.weight != nullptr)
          p.c.weight[at] = p.score == nullptr ? 0.f : p.score[static_cast<int64_t>(h) * p.total_tokens + s0 + first + i];
      }
    }
    ++rank;
  }
  if (p1 == L && tid == 0) {
    p.c.count[row] = min(before + total, p.c.capacity);
    if (p.c.seen != nullptr) p.c.seen[row] = L;
  }
  __syncthreads();
  const int64_t stride = static_cast<int64_t>(p.c.n_kv_heads) * D;
  copy_rows<D, kF8, kPcThreads, kF8 ? 4 : 8>(p.c, p.k + s0 * stride, p.v + s0 * stride, stride, h, list, n);
}

cudaError_t launch_paged_compact(PagedCompactParams& p, int head_dim, bool f8, cudaStream_t stream) {
  int longest = 1;
  for (int b = 0; b < p.c.batch; ++b) longest = std::max(longest, p.start[b + 1] - p.start[b]);
  // Short blocks keep the CTAs many and even; the conversion to e4m3 has more to do per row and takes 512 positions
  // (8 prompts of 100,003 tokens in all, e4m3: 80 us with 512, 82 with 256; bf16: 85 and 83.5, 99% of the copy
  // bandwidth).  Beyond 32,768 tokens counting the mask again 4 times as often would show.
  p.block = longest > 32768 ? kPcMaxBlock : f8 ? 512 : 256;
  const dim3 grid(p.c.batch * p.c.n_kv_heads, (longest + p.block - 1) / p.block), block(kPcThreads);
  if (head_dim == 128)
    return f8 ? launch_paged(paged_compact_kernel<128, true>, grid, block, 0, 1, stream, p)
              : launch_paged(paged_compact_kernel<128, false>, grid, block, 0, 1, stream, p);
  return f8 ? launch_paged(paged_compact_kernel<64, true>, grid, block, 0, 1, stream, p)
            : launch_paged(paged_compact_kernel<64, false>, grid, block, 0, 1, stream, p);
}

}  // namespace kvpop
