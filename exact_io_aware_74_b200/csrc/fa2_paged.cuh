// Tables of a serving step and the write into the paged cache.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace fa2 {

// ------------------------------------------------------------------------------------
// tables
// ------------------------------------------------------------------------------------

struct TablesParams {
  const int* context_lens;
  const int* new_lens;
  const int* free_blocks;
  int* block_table;
  int* cu_seqlens;
  int* seq_lens;
  int* positions;
  int* slots;
  int* used;
  int num_free, B, T, block_size, max_blocks;
};

constexpr int kTablesThreads = 512;

// Blocks that hold n >= 0 tokens; n + bs - 1 may pass 2^31.
__device__ __forceinline__ int blocks_for(int n, int bs) { return n > 0 ? (n - 1) / bs + 1 : 0; }

// Every CTA sums the lengths of all requests (a block scan per 512 of them) and then
// writes the table rows of every gridDim-th request and the slots of its own stretch
// of tokens.  No CTA waits for another: a slot whose block is new in this step is taken
// from the free list again rather than from the table entry that another CTA writes.
// A step of 64 single tokens takes 5 us, 500 requests that bring 0.67 M tokens 15 us (B200): the
// chain of loads, the scan and each token's search, not the 5.7 MB; a call from Python takes 17
// us, the host's time.
// Sums past 2^31 give unspecified tables, but every index below is checked or clamped, so
// that none reads or writes outside them.
__global__ void __launch_bounds__(kTablesThreads)
fa2_paged_tables_kernel(const TablesParams p) {
  __shared__ int s_ctx[kTablesThreads], s_cu[kTablesThreads + 1], s_first[kTablesThreads];
  __shared__ int w_new[kTablesThreads / 32], w_take[kTablesThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_cta = (p.T + gridDim.x - 1) / gridDim.x;
  const int t_lo = min(p.T, static_cast<int>(blockIdx.x) * per_cta), t_hi = min(p.T, t_lo + per_cta);
  const int bs = p.block_size;
  int cu0 = 0, take0 = 0;  // sums over the requests before this batch of 512
  for (int r0 = 0; r0 < p.B; r0 += kTablesThreads) {
    const int r = r0 + tid;
    const int ctx = r < p.B ? max(0, p.context_lens[r]) : 0;
    const int nw = r < p.B ? min(max(0, p.new_lens[r]), 0x7fffffff - ctx) : 0;
    const int had = blocks_for(ctx, bs), need = blocks_for(ctx + nw, bs);
    int a = nw, b = need - had;  // inclusive sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) a += x, b += y;
    }
    if (lane == 31) w_new[warp] = a, w_take[warp] = b;
    __syncthreads();
    int ba = cu0, bb = take0, ta = 0, tb = 0;
    for (int w = 0; w < kTablesThreads / 32; ++w) {
      if (w < warp) ba += w_new[w], bb += w_take[w];
      ta += w_new[w];
      tb += w_take[w];
    }
    a += ba;
    b += bb;
    s_ctx[tid] = ctx;
    s_cu[tid] = a - nw;
    if (tid == kTablesThreads - 1) s_cu[kTablesThreads] = a;
    s_first[tid] = b - (need - had) - had;  // free-list place of block i: s_first + i
    if (blockIdx.x == 0 && r < p.B) {
      p.cu_seqlens[r] = a - nw;
      p.seq_lens[r] = ctx + nw;
      if (r == p.B - 1) {
        p.cu_seqlens[p.B] = a;
        *p.used = b;
      }
    }
    __syncthreads();
    const int cnt = min(kTablesThreads, p.B - r0);
    // Table rows: a warp to a request, every gridDim-th of them here.
    for (int i = warp; i < cnt; i += kTablesThreads / 32) {
      if ((r0 + i) % static_cast<int>(gridDim.x) != static_cast<int>(blockIdx.x)) continue;
      const int c = s_ctx[i], n = min(max(s_cu[i + 1] - s_cu[i], 0), 0x7fffffff - c);
      const int h = blocks_for(c, bs), e = min(p.max_blocks, blocks_for(c + n, bs));
      int* row = p.block_table + static_cast<size_t>(r0 + i) * p.max_blocks;
      for (long long k = static_cast<long long>(h) + lane; k < e; k += 32) {  // (h + lane may pass 2^31)
        const int f = s_first[i] + static_cast<int>(k);
        row[k] = f >= 0 && f < p.num_free ? p.free_blocks[f] : -1;
      }
    }
    // Tokens of this CTA's stretch that belong to these requests.
    const int lo = min(t_hi, max(t_lo, cu0)), hi = min(t_hi, cu0 + ta);
    for (int t = lo + tid; t < hi; t += kTablesThreads) {
      int i = 0, j = cnt;  // the last request that starts at or before t
      while (j - i > 1) {
        const int m = (i + j) >> 1;
        if (s_cu[m] <= t) i = m; else j = m;
      }
      const int c = s_ctx[i], pos = c + t - s_cu[i];
      const int k = pos / bs;
      int block = -1;
      if (pos >= 0 && k < p.max_blocks) {
        if (k < blocks_for(c, bs)) {
          block = p.block_table[static_cast<size_t>(r0 + i) * p.max_blocks + k];
        } else {
          const int f = s_first[i] + k;
          if (f >= 0 && f < p.num_free) block = p.free_blocks[f];
        }
      }
      p.positions[t] = pos;
      p.slots[t] = block < 0 || block > 0x7fffffff / bs - 1 ? -1 : block * bs + pos - k * bs;
    }
    cu0 += ta;
    take0 += tb;
    __syncthreads();  // the shared sums are rewritten
  }
  for (int t = min(t_hi, max(t_lo, cu0)) + tid; t < t_hi; t += kTablesThreads) {
    p.positions[t] = 0;
    p.slots[t] = -1;
  }
}

// ------------------------------------------------------------------------------------
// append
// ------------------------------------------------------------------------------------

struct AppendParams {
  const uint16_t* src[2];
  uint16_t* dst[2];
  long long src_row[2], src_head[2], dst_block[2], dst_head[2], dst_row[2];
  const int* slots;
  unsigned int* status;
  int T, Hkv, vec, num_blocks, block_size;  // vec: 16-byte pieces of a head
};

// A thread keeps its 16 bytes of the row (its head and column are found once) and copies
// them for kAppendRows rows, the loads of all before the first store: the copy is bound by
// HBM, and with a division per 16 bytes and one load in flight a thread it took 104 us for
// 55k rows of 8 heads of 128 (69 us at the copy rate; B200).  blockIdx.y: keys or values,
// and the piece of the row where it has more than kAppendThreads.
constexpr int kAppendThreads = 512, kAppendRows = 4;

__global__ void __launch_bounds__(kAppendThreads) fa2_paged_append_kernel(const AppendParams p) {
  const int w = blockIdx.y & 1, x = (blockIdx.y >> 1) * blockDim.x + threadIdx.x;
  if (x >= p.Hkv * p.vec) return;
  const int h = x / p.vec, c = x - h * p.vec;
  const uint16_t* src = p.src[w] + h * p.src_head[w] + c * 8;
  uint16_t* dst = p.dst[w] + h * p.dst_head[w] + c * 8;
  const int t0 = blockIdx.x * (kAppendRows * blockDim.y) + threadIdx.y;
  int slot[kAppendRows];
  uint4 v[kAppendRows];
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int t = t0 + i * blockDim.y;
    slot[i] = t < p.T ? p.slots[t] : -1;
    if (slot[i] >= 0) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + t * p.src_row[w]));
  }
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    if (slot[i] < 0) continue;
    const int block = static_cast<unsigned int>(slot[i]) / static_cast<unsigned int>(p.block_size);
    const int pos = slot[i] - block * p.block_size;
    if (block >= p.num_blocks) {
      if (x == 0) atomicCAS(p.status, 0u, kStatusInvalid | (kPSiteSlot << 8));
      continue;
    }
    *reinterpret_cast<uint4*>(dst + block * p.dst_block[w] + pos * p.dst_row[w]) = v[i];
  }
}

}  // namespace fa2
