// Forward attention over packed sequences and over paged caches, with grouped heads.
//
// The tiles, the online softmax and the products are those of the dense forward
// (fa2_fwd.cuh): 128 x 128 score tiles in tensor memory, one thread to a score row, P
// back to tensor memory for P V, the lazy rescale.  What differs:
//
// Rows.  A query tile holds the G = H / Hkv query heads of one key/value head: row
// r = token * G + head, 128 / G tokens to a tile.  The K and V of a tile are then read
// once for all the heads that share them, and a single token still fills G rows.
//
// Items.  An item is one (sequence, key/value head, QT tiles of rows) and a range of
// key tiles.  The lengths are on the device, so the items are found there:
//   packed:  the grid has one CTA for every item there could be (T / rows + B, times
//            heads); a running CTA takes over the items of CTAs that have not started
//            (cluster launch control), so that the hardware's block scheduler hands out
//            the items in order of their index, heaviest first, and no counter in
//            memory is needed.
//   paged:   the key tiles of all items, end to end, are cut into equal shares, one per
//            CTA.  An item that is cut leaves float partials, which a second kernel
//            merges; an item inside one share is written directly.  A decode step of any
//            mix of lengths then keeps every SM streaming until the end.
//
// Roles (384 threads, three warpgroups):
//   warps 0-3, 4-7  softmax of tile 0 and tile 1 (QT = 1: warps 4-7 idle)
//   warp 8          Q and K tiles by TMA; pages one box each
//   warp 9          MMA issuer (one thread; few rows: scheduler and issuer of S)
//   warp 10         (few rows: issuer of P V) scheduler: finds the CTA's next item while the current one runs
//   warp 11         V tiles by TMA; zeroes the rows that belong to no visible key (a sequence
//                   that ends inside a tile), so that nothing there, NaN included, reaches P V
// The CTA runs its items as one stream: the rings of Q, K and V tiles and every barrier's
// phase go on across items, the first scores of the next item are issued right behind
// the last P V of this one, and its epilogue overlaps them.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace fa2 {

struct SeqParams {
  uint16_t* O;
  long long o_row, o_head;  // strides in elements
  float* LSE;               // [H][T]
  const int* cu;            // [B + 1]
  const int* seq_lens;      // paged: [B]
  const int* block_table;   // paged: [B][max_blocks]
  float* O_part;            // [2 grid][QT * 128][D]
  float* LSE_part;          // [2 grid][QT * 128]
  int4* merge;              // [grid]: the cut block that starts in the share (row, tokens, head, parts)
  unsigned int* status;
  unsigned long long wait_ns;
  int B, T, Hkv, G, d, tpt;  // tpt: tokens to a tile, 128 / G
  int causal, window, fault, head_group;
  int num_blocks, block_size, max_blocks;
  int box_shift, tiles_block;  // paged: rows of a box, min(block_size, 128), are 1 << box_shift; key tiles to a block
  float scale_log2;
};

// NQ = 0: the layout above.  NQ = 16 (QT = 1): items of at most NQ rows, with the
// operands of both products swapped (see the few-rows roles of the kernel).
template <int D_, int QT_, int NQ_ = 0>
struct SeqCfg {
  static constexpr int D = D_, QT = QT_, NQ = NQ_;
  static_assert(QT == 1 || D <= 128, "two accumulators fit tensor memory up to D = 128");
  static_assert(NQ == 0 || (QT == 1 && D <= 128 && NQ == 16), "few rows");
  static constexpr int KCH = D / 64;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int QCHUNK = NQ ? NQ * 128 : CHUNK, QTILE = KCH * QCHUNK;
  // Ring stages within 227 KB (tiles of 16, 32, 48, 64 KB).  Two query tiles have a third
  // slot at D = 128, so that the next item's first tile loads during this one.
  static constexpr int QS = NQ ? 2 : (D == 64 ? 4 : (D == 128 ? (QT == 2 ? 3 : 2) : 1));
  // (Few rows: as many S blocks as K slots; with V slots in even number a product's barrier
  // releases its slot too, see the issuer.  Three slots each at D = 128: 4 and 2 took 275, not
  // 264 us for 64 requests over 6k tokens in blocks of 64, B200.)
  static constexpr int KS = NQ ? (D == 64 ? 6 : 3) : (D == 64 ? 4 : (D == 256 ? 1 : 2));
  static constexpr int VS = NQ ? (D == 64 ? 6 : 3) : (D == 64 ? 4 : (D == 128 ? (QT == 2 ? 2 : 3) : 1));
  // Few rows: P^T of each warpgroup, two chunks of 64 keys, PB buffers each (with two a
  // warpgroup need not wait for its last product before it writes the next P).  (At D = 64 the V operand's
  // upper 64 rows are whatever lies 16 KB behind the tile: at least that much follows.)
  static constexpr int PBUF = 2 * NQ * 128, PB = D == 64 ? 2 : 1;
  static constexpr bool SHARE_V = NQ && VS % 2 == 0;
  static_assert(NQ == 0 || PB == 1 || (SHARE_V && 2 * PB <= VS), "a product's barrier comes round after its P buffer");
  static constexpr int PREST = QS * QTILE + 2 * PB * PBUF;
  static constexpr int REST = NQ ? (PREST < CHUNK ? CHUNK : PREST) : QS * TILE;
  static constexpr int SMEM = (KS + VS) * TILE + REST + 1024;
  static_assert(SMEM <= 226 * 1024, "shared memory");
  static constexpr int THREADS = 384;
  static constexpr int LAUNCH_REGS = 168;
  static constexpr int SOFT_REGS = 216, OTHER_REGS = 72;
  static_assert(2 * 128 * SOFT_REGS + 128 * OTHER_REGS <= THREADS * LAUNCH_REGS, "register re-split");
  __host__ __device__ static constexpr uint32_t O_COL(int t) { return 256u + t * (NQ ? NQ : D); }
  // D = 64 with two tiles: P in columns of its own (the next scores overwrite S early).
  static constexpr bool SEP = D == 64 && QT == 2;
  __host__ __device__ static constexpr uint32_t P_COL(int t) { return 384u + 64u * t; }
};

enum SeqSite : uint32_t {
  kQSiteItem = 80, kQSiteItemEmpty, kQSiteProd, kQSiteMmaQ, kQSiteMmaK, kQSiteMmaV, kQSiteMmaP, kQSiteMmaO,
  kQSiteMmaDrain, kQSiteSoftS, kQSiteSoftO, kQSiteClc, kQSiteDrain
};

constexpr int kSeqItems = 4;  // ring of items handed to the roles
constexpr int kHeld = 256;    // sequences whose counts a scheduling warp keeps in shared memory

struct SeqItem {
  int row0, n_tok;   // first packed query row, tokens
  int kvh;           // key/value head
  int key0;          // packed: row of the sequence's first key; paged: the request
  int nk, first;     // keys of the sequence; first one that any row of the item sees
  int pos;           // position of the item's first token among the keys
  int lo[2], hi[2];  // key tiles of each query tile
  int j0, n;         // key tiles of the item: j0 .. j0 + n - 1
  int part;          // partial slot, -1: O and LSE are written
  int valid;
  int pad;
};

// ------------------------------------------------------------------------------------
// items
// ------------------------------------------------------------------------------------

struct SeqLen {
  int row0, n, nk;
};

template <bool PAGED>
__device__ __forceinline__ SeqLen seq_len(const SeqParams& p, int b) {
  SeqLen s;
  s.row0 = min(max(p.cu[b], 0), p.T);
  s.n = min(max(p.cu[b + 1], s.row0), p.T) - s.row0;
  s.nk = s.n;
  if (PAGED) s.nk = min(max(p.seq_lens[b], 0), p.max_blocks * p.block_size);
  return s;
}

// Key tiles that tokens [a, e) of a sequence need; the same for the whole item.
__device__ __forceinline__ void key_range(const SeqParams& p, const SeqLen& s, int a, int e, int& lo, int& hi) {
  const int pos = s.nk - s.n;  // of token 0
  lo = hi = 0;
  if (a >= e) return;
  const int last = p.causal ? min(pos + e - 1, s.nk - 1) : s.nk - 1;
  hi = last >= 0 ? (last >> 7) + 1 : 0;
  if (p.window > 0) lo = max(0, pos + a - p.window + 1) >> 7;
  if (hi <= lo) lo = hi = 0;
}

template <bool PAGED, int QT>
__device__ __forceinline__ void make_item(const SeqParams& p, const SeqLen& s, int b, int kvh, int blk, SeqItem& it) {
  const int a = blk * (QT * p.tpt), e = min(s.n, a + QT * p.tpt), m = min(e, a + p.tpt);
  it.row0 = s.row0 + a;
  it.n_tok = e - a;
  it.kvh = kvh;
  it.key0 = PAGED ? b : s.row0;
  it.nk = s.nk;
  it.pos = s.nk - s.n + a;
  it.first = p.window > 0 ? max(0, it.pos - p.window + 1) : 0;
  key_range(p, s, a, m, it.lo[0], it.hi[0]);
  it.lo[1] = it.hi[1] = 0;
  if (QT == 2) key_range(p, s, m, e, it.lo[1], it.hi[1]);
  const bool h0 = it.hi[0] > 0, h1 = it.hi[1] > 0;
  it.j0 = h0 ? (h1 ? min(it.lo[0], it.lo[1]) : it.lo[0]) : it.lo[1];
  it.n = max(it.hi[0], it.hi[1]) - it.j0;
  it.part = -1;
  it.valid = 1;
}

// The item cut to the key tiles [a, e) counted from its first one.
__device__ __forceinline__ void cut_item(SeqItem& it, int a, int e) {
  const int s = it.j0 + a, f = it.j0 + e;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.lo[t] = max(it.lo[t], s);
    it.hi[t] = min(it.hi[t], f);
    if (it.hi[t] <= it.lo[t]) it.lo[t] = it.hi[t] = 0;
  }
  const bool h0 = it.hi[0] > 0, h1 = it.hi[1] > 0;
  it.j0 = h0 ? (h1 ? min(it.lo[0], it.lo[1]) : it.lo[0]) : it.lo[1];
  it.n = max(it.hi[0], it.hi[1]) - it.j0;
}

// Units of work of block blk of a sequence: its key tiles (both query tiles' together, at
// least one) and IU for its start and end, which come first in the linear order.  (With key
// tiles alone the share with a prompt's many short blocks ended at 300 us, the others at 175;
// the shares of a decode step ended between 180 and 233 us with one unit to an item.)
constexpr int kItemUnits = 4;
template <int QT, int IU>
__device__ __forceinline__ int block_units(const SeqParams& p, int n, int nk, int blk) {
  const int a = blk * (QT * p.tpt);
  int lo, hi;
  key_range(p, SeqLen{0, n, nk}, a, min(n, a + QT * p.tpt), lo, hi);
  return max(1, hi - lo) + IU;
}
__device__ __forceinline__ int blocks_of(int n, int R) { return n <= R ? (n > 0) : (n + R - 1) / R; }

// Units of one key/value head of a sequence per lane: of a single block each lane its own,
// of more the whole warp together.
template <int QT, int IU>
__device__ __forceinline__ int lane_units(const SeqParams& p, int n, int nk, int lane) {
  const int R = QT * p.tpt;
  int u = n > 0 ? block_units<QT, IU>(p, n, nk, 0) : 0;
  unsigned int many = __ballot_sync(0xffffffffu, n > R);
#pragma unroll 1
  while (many) {
    const int l = __ffs(many) - 1;
    many &= many - 1;
    const int on = __shfl_sync(0xffffffffu, n, l), ok = __shfl_sync(0xffffffffu, nk, l);
    int part = 0;
#pragma unroll 1
    for (int i = lane; i * R < on; i += 32) part += block_units<QT, IU>(p, on, ok, i);
    part = __reduce_add_sync(0xffffffffu, part);
    if (lane == l) u = part;
  }
  return u;
}

__device__ __forceinline__ int warp_inclusive(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Units to a share: equal for `grid` CTAs (the last ones may get fewer or none), at least
// kMinUnits.  All units together are below 2^31 (checked by the caller): 64-bit divisions
// alone were 7 KB of code.
constexpr int kMinUnits = 2;
__device__ __forceinline__ int share_units(int total, int grid) {
  return max((static_cast<unsigned int>(total) + grid - 1) / static_cast<unsigned int>(grid), kMinUnits + 0u);
}

// The linear order of the units: sequence, head, block, key tile.  Whole warp.
struct UnitAt {
  int b, kvh, blk, at;  // at: units of the block before x
  SeqLen s;
};

// Finds share c: units x .. xe - 1, `per` to a share.  False when there is none.  held:
// kHeld ints of shared memory.  One loop body serves the total and the search.
template <int QT, int IU>
__device__ __forceinline__ bool find_share(const SeqParams& p, int grid, int c, int* held, int lane, int& per, int& x, int& xe,
                                           UnitAt& r) {
  int total = 0, rem = 0;
  int units = 1;  // of one head of the sequence found
  r.b = -1;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int v;
      if (pass == 1 && b0 < kHeld) {
        v = held[b0 + lane];
      } else {
        SeqLen s{0, 0, 0};
        if (b0 + lane < p.B) s = seq_len<true>(p, b0 + lane);
        v = lane_units<QT, IU>(p, s.n, s.nk, lane);
        if (b0 < kHeld) held[b0 + lane] = v;
      }
      const int inc = warp_inclusive(v, lane);
      const int end = inc * p.Hkv;
      if (pass == 0) {
        total += __shfl_sync(0xffffffffu, end, 31);
        continue;
      }
      const unsigned int m = __ballot_sync(0xffffffffu, end > rem);
      if (m) {
        const int l = __ffs(m) - 1;
        r.b = b0 + l;
        units = __shfl_sync(0xffffffffu, v, l);
        rem -= __shfl_sync(0xffffffffu, end, l) - units * p.Hkv;
        break;
      }
      rem -= __shfl_sync(0xffffffffu, end, 31);
    }
    if (pass == 0) {
      per = share_units(total, grid);
      x = rem = per * c;
      if (x >= total || x < 0) return false;  // (per * c may pass 2^31)
      xe = min(total - x, per) + x;
      __syncwarp();
    }
  }
  if (r.b < 0) return false;  // (offsets that fall can hold more rows than T, and the sums wrap)
  r.s = seq_len<true>(p, r.b);
  r.kvh = static_cast<unsigned int>(rem) / static_cast<unsigned int>(units);
  if (static_cast<unsigned int>(r.kvh) >= static_cast<unsigned int>(p.Hkv)) return false;  // (likewise)
  int at = rem - r.kvh * units;
  const int R = QT * p.tpt, nb = blocks_of(r.s.n, R);
  r.blk = 0;
  if (nb > 1) {
#pragma unroll 1
    for (int i0 = 0; i0 < nb; i0 += 32) {
      const int v = i0 + lane < nb ? block_units<QT, IU>(p, r.s.n, r.s.nk, i0 + lane) : 0;
      const int inc = warp_inclusive(v, lane);
      const unsigned int m = __ballot_sync(0xffffffffu, inc > at);
      if (m) {
        const int l = __ffs(m) - 1;
        r.blk = i0 + l;
        at -= __shfl_sync(0xffffffffu, inc - v, l);
        break;
      }
      at -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  r.at = at;
  return true;
}

// The items of one CTA's share, one after the other.  Whole warp.
template <int QT, int IU>
struct ShareWalk {
  int per, x, xe;  // units to a share; next unit, end
  UnitAt u;

  __device__ __forceinline__ void start(const SeqParams& p, int* held, int lane) {
    const int c = blockIdx.x;
    if (lane == 0) p.merge[c] = make_int4(0, 0, 0, 0);  // nothing to merge, until a block is cut
    if (!find_share<QT, IU>(p, gridDim.x, c, held, lane, per, x, xe, u)) x = xe = 0;
  }
  // The next item with key tiles; false at the end of the share.
  __device__ __forceinline__ bool next(const SeqParams& p, int lane, SeqItem& it) {
    const int c = blockIdx.x, R = QT * p.tpt;
    bool found = false;
#pragma unroll 1
    while (!found && x < xe) {
      const int len = block_units<QT, IU>(p, u.s.n, u.s.nk, u.blk);
      const int take = min(len - u.at, xe - x);
      make_item<true, QT>(p, u.s, u.b, u.kvh, u.blk, it);
      // Key tiles [a, e) of the block's fall into this share.
      const int a = max(0, u.at - IU), e = max(0, u.at + take - IU);
      if (it.n == 0) {
        // Rows that see no key: O = 0 and LSE = -inf, here.  (The other roles then never meet
        // an item without key tiles, which would be in the way of the next one.)
        if (e > a)
#pragma unroll 1
          for (int r = 0; r < it.n_tok * p.G; ++r) {
            const int row = it.row0 + r / p.G, head = u.kvh * p.G + r % p.G;
            if (lane * 8 < p.d)
              *reinterpret_cast<uint4*>(p.O + row * p.o_row + head * p.o_head + lane * 8) = make_uint4(0, 0, 0, 0);
            if (lane == 0) p.LSE[static_cast<size_t>(head) * p.T + row] = -INFINITY;
          }
      } else if (e > a) {
        found = true;
        if (a > 0 || e < len - IU) {
          if (a == 0 && lane == 0) {
            // The block goes on in the next shares: for the merge kernel.
            int parts = 1;
#pragma unroll 1
            for (int left = x + len - u.at - xe; left > 0; left -= per) ++parts;
            p.merge[c] = make_int4(it.row0, it.n_tok, u.kvh, parts);
          }
          cut_item(it, a, e);
          it.part = 2 * c + (a > 0 ? 0 : 1);
        }
      }
      x += take;
      if (x >= xe) break;
      u.at = 0;
      if (++u.blk * R >= u.s.n) {
        u.blk = 0;
        if (++u.kvh >= p.Hkv) {
          u.kvh = 0;
          do {
            if (++u.b >= p.B) break;  // (likewise: units are left otherwise)
            u.s = seq_len<true>(p, u.b);
          } while (u.s.n == 0);
          if (u.b >= p.B) x = xe;
        }
      }
    }
    return found;
  }
};

__device__ __forceinline__ int rows_of(const int* cu, int T, int b) {
  const int s = min(max(cu[b], 0), T);
  return min(max(cu[b + 1], s), T) - s;
}

// Packed: the order of the items, found by one warp.  Up to CAP sequences their block
// counts are kept in shared memory, and the order is head group by head group, in a group
// the blocks of the highest level (index from the sequence's start) of all sequences first,
// heads innermost: heaviest first, when causal.  With more sequences the blocks lie
// sequence by sequence, highest first (cu[b] / R + b is where sequence b's start: its last
// block may be partial, so some places hold none).  Searching the counts in global memory
// for the first order took 5 to 9 us an item with 148 and 740 sequences (B200).
struct BlockAt {
  int b, level, kvh;
};

template <int CAP>  // sequences whose counts fit
struct BlockOrder {
  int* held;
  int n_blocks, max_blk;  // of one head; of one sequence

  __device__ __forceinline__ void load(int* shared, const int* cu, int B, int T, int R, int lane) {
    held = shared;
    max_blk = 0;
    n_blocks = T / R + B;
    if (B > CAP) return;
    int sum = 0, most = 0;
#pragma unroll 2
    for (int b = lane; b < B; b += 32) {
      const int n = (rows_of(cu, T, b) + R - 1) / R;
      held[b] = n;
      sum += n;
      most = max(most, n);
    }
    n_blocks = min(static_cast<int>(__reduce_add_sync(0xffffffffu, sum)), T / R + B);  // (bad offsets: no more)
    max_blk = __reduce_max_sync(0xffffffffu, most);
    __syncwarp();
  }
  // Item w (whole warp); false when the place holds none.
  __device__ __forceinline__ bool find(const int* cu, int B, int T, int Hkv, int head_group, int R, int w, int lane,
                                       BlockAt& r) const {
    if (w >= static_cast<long long>(n_blocks) * Hkv) return false;
    const int per = head_group * n_blocks, grp = w / per, at = w - grp * per;
    const int heads = min(head_group, Hkv - grp * head_group);
    const int rank = at / heads;
    r.kvh = grp * head_group + at - rank * heads;
    if (B > CAP) {
      int lo = 0, n = B;  // the last sequence whose place is at or before rank is in [lo, lo + n)
#pragma unroll 1
      while (n > 1) {
        const int step = (n + 31) / 32, b = lo + lane * step;
        const bool le = lane * step < n && min(max(cu[b], 0), T) / R + b <= rank;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        lo += k * step;
        n = min(step, n - k * step);
      }
      r.b = lo;
      const int blocks = (rows_of(cu, T, lo) + R - 1) / R;
      r.level = blocks - 1 - (rank - (min(max(cu[lo], 0), T) / R + lo));
      return r.level >= 0 && r.level < blocks;
    }
    // The largest level with more than `rank` blocks at that level and above, by bisection;
    // `above`: the blocks above it.
    int lo = 0, hi = max_blk, above = 0;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      int c = 0;
#pragma unroll 2
      for (int b = lane; b < B; b += 32) c += max(0, held[b] - mid);
      c = __reduce_add_sync(0xffffffffu, c);
      if (c > rank) lo = mid; else hi = mid, above = c;
    }
    r.level = lo;
    int i = rank - above;  // the i-th sequence with more than lo blocks
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      const bool has = b0 + lane < B && held[b0 + lane] > lo;
      const unsigned int m = __ballot_sync(0xffffffffu, has);
      const unsigned int hit = __ballot_sync(0xffffffffu, has && __popc(m & ((1u << lane) - 1u)) == i);
      if (hit) {
        r.b = b0 + __ffs(hit) - 1;
        return true;
      }
      i -= __popc(m);
    }
    return false;
  }
};

// ------------------------------------------------------------------------------------
// cluster launch control: the index of a CTA of this grid that has not started
// ------------------------------------------------------------------------------------

__device__ __forceinline__ void clc_try_cancel(uint4* response, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(response)),
      "r"(smem_u32(bar))
      : "memory");
}

// The cancelled CTA's blockIdx.x, or -1 when none was left.
__device__ __forceinline__ int clc_index(const uint4* response) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(response))
      : "memory");
  return ok ? static_cast<int>(x) : -1;
}

// 4-D tiled load (a page's rows of one head).
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// ------------------------------------------------------------------------------------
// the kernel
// ------------------------------------------------------------------------------------

// mbar_wait with its loop out of line, for the roles off the critical path (with it in the
// MMA issuer the not causal 2 x 32 x 8192 forward took 2590 us, not 2250): some thirty
// copies of the loop are a quarter of the kernel's code, and what runs once an item then
// misses the instruction cache (238 KB of code ran items of one key tile at 11 us, 127 KB at
// 7 us; B200).  For the same reason what runs once an item or seldom is not unrolled: on SMs
// that had been through a few items, straight arithmetic of the softmax stalled for up to 2 us
// a key tile.  With 88 instead of 112 KB (and 92 instead of 153 for few rows) a step of chunks
// over 8k caches takes 195 us, not 227, the full decode step 219, not 232.
static __device__ __noinline__ bool mbar_wait_loop(uint32_t bar, uint32_t parity, unsigned int* status,
                                                   volatile int* abort, uint64_t limit_ns, uint32_t site) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 15u) == 0u) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        report_timeout(WaitCtl{status, abort, limit_ns}, site);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool mbar_wait_far(uint64_t* bar, uint32_t parity, const WaitCtl& w, uint32_t site) {
  if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_loop(smem_u32(bar), parity, w.status, w.abort, w.limit_ns, site);
}

// Keys of tile j that some row of the item sees, counted from the tile's first key.
__device__ __forceinline__ void tile_keys(const SeqItem& it, int j, int& a, int& e) {
  a = max(it.first - j * 128, 0);
  e = min(it.nk - j * 128, 128);
}

template <int D, bool BF16, int QT, bool PAGED, int NQ>
__global__ void __launch_bounds__(384, 1)
fa2_seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const SeqParams p) {
  using C = SeqCfg<D, QT, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::KS * C::TILE;
  uint8_t* sQ = sV + C::VS * C::TILE;
  [[maybe_unused]] uint8_t* sP = sQ + C::QS * C::QTILE;  // few rows: P^T, one buffer to a warpgroup

  __shared__ __align__(16) uint4 clc_response;
  constexpr int NI = kSeqItems;
  __shared__ __align__(16) SeqItem items[NI];
  __shared__ uint64_t item_full[NI], item_empty[NI], clc_full;
  __shared__ uint64_t q_full[C::QS], q_empty[C::QS], k_full[C::KS], k_empty[C::KS];
  __shared__ uint64_t v_full[C::VS], v_empty[C::VS], v_raw[C::VS];
  __shared__ uint64_t s_full[6], s_free[6], p_ready[4], o_done[6], o_free[2], drain, drain_pv;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int held[kHeld];  // the scheduling warp's

  griddep_launch_dependents();  // the merge kernel waits for this grid before it reads

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  WaitCtl wc{p.status, &abort_flag, p.wait_ns};

  if (threadIdx.x == 8 * 32) {
    abort_flag = 0;
    for (int i = 0; i < NI; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], NQ ? 12 : 3 + 4 * QT);  // two producers, the issuers and the softmax warps
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_ready[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&o_free[i], NQ ? 8 : 4);
    }
    mbar_init(&clc_full, 1);
    for (int i = 0; i < C::QS; ++i) { mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1); }
    for (int i = 0; i < C::KS; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < C::VS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_raw[i], 1);
    }
    mbar_init(&drain, 1);
    mbar_init(&drain_pv, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;

  if (warp >= 8) {
    regs_dec<C::OTHER_REGS>();
    if (NQ == 0 && warp == 10) {
      // ---------------------------------------------------------------- scheduler
      int ii = 0;
      auto publish = [&](const SeqItem& it) -> bool {
        const int s = ii % NI;
        bool ok = true;
        if (ii >= NI) ok = mbar_wait_far(&item_empty[s], ((ii / NI) - 1) & 1, wc, kQSiteItemEmpty);
        if (!__all_sync(0xffffffffu, ok)) return false;
        if (lane == 0) {
          items[s] = it;
          mbar_arrive(&item_full[s]);
        }
        ++ii;
        return true;
      };
      SeqItem it{};
      bool ok = true;
      if constexpr (PAGED) {
        ShareWalk<QT, kItemUnits> walk;
        walk.start(p, held, lane);
        while (ok && walk.next(p, lane, it)) ok = publish(it);
      } else {
        const int R = QT * p.tpt;
        BlockOrder<kHeld> order;
        order.load(held, p.cu, p.B, p.T, R, lane);
        BlockAt at;
        int w = blockIdx.x;
        for (int k = 0; ok && w >= 0; ++k) {
          if (order.find(p.cu, p.B, p.T, p.Hkv, p.head_group, R, w, lane, at)) {
            make_item<false, QT>(p, seq_len<false>(p, at.b), at.b, at.kvh, at.level, it);
            ok = publish(it);
          }
          // The next index only once the item before this one is done with: a CTA holds
          // at most one item that it has not begun.
          if (ok && ii >= 2)
            ok = __all_sync(0xffffffffu, mbar_wait_far(&item_empty[(ii - 2) % NI], ((ii - 2) / NI) & 1, wc, kQSiteItemEmpty));
          if (!ok) break;
          if (lane == 0) {
            fence_proxy_async_smem();  // the response was read before it is written again
            mbar_arrive_expect_tx(&clc_full, 16);
            clc_try_cancel(&clc_response, &clc_full);
          }
          __syncwarp();
          volatile int no_abort = 0;  // the response always lands before the CTA leaves
          WaitCtl cw{p.status, &no_abort, p.wait_ns};
          ok = __all_sync(0xffffffffu, mbar_wait_far(&clc_full, k & 1, cw, kQSiteClc));
          if (!ok) break;
          w = lane == 0 ? clc_index(&clc_response) : 0;
          w = __shfl_sync(0xffffffffu, w, 0);
        }
      }
      it.valid = 0;
      if (ok) publish(it);
    } else if (warp == 8 || warp == 11) {
      // ---------------------------------------------------------------- producers
      // Warp 8 loads the Q and K tiles, warp 11 the V tiles, each in the order in which the MMA
      // issuer takes them.  (A page of 16 positions is 2 KB to a box: one warp issuing the
      // boxes of both held a decode step to 3.8 TB/s.)  Warp 11 also zeroes the V rows that no
      // row of the item sees, once such a tile has landed (on v_raw; v_full is then its own).
      const bool is_v = warp == 11;
      [[maybe_unused]] const uint64_t keep = policy_evict_last();
      const CUtensorMap* map = is_v ? &tmV : &tmK;
      uint8_t* ring = is_v ? sV : sK;
      const int slots = is_v ? C::VS : C::KS;
      uint64_t* full = is_v ? v_full : k_full;
      // Few rows: a product's completion barrier is its slot's release too.
      uint64_t* empty = is_v ? (C::SHARE_V ? o_done : v_empty) : (NQ ? s_full : k_empty);
      int qc = 0, slot = 0;              // Q tiles loaded; this warp's next slot
      unsigned int turn = 0;             // parity of the turn around the ring
      bool round = false;                // the ring has been around once
      unsigned int raw_par = 0;          // V: parity of the loads on v_raw, per slot
      int fix = -1, fix_a = 0, fix_e = 0;  // V: slot to be zeroed outside rows [fix_a, fix_e)
      bool ok = true, skip = p.fault == 1 && !is_v;  // test hook: the first K tile is not loaded
      [[maybe_unused]] const int bsh = p.box_shift, nbox = 128 >> bsh;  // rows of a box: 1 << bsh
      auto wait_all = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_wait_far(bar, par, wc, kQSiteProd)) != 0;
      };
      // Lane i: the page of box i of tile j (read a tile ahead of its loads).
      auto pages_of = [&](const SeqItem& it, int j) -> int {
        int a, e, pg = 0;
        tile_keys(it, j, a, e);
        if (lane < nbox && lane << bsh < e && (lane + 1) << bsh > a) {
          const int at = p.tiles_block <= 1 ? j * nbox + lane : j / p.tiles_block;
          pg = p.block_table[static_cast<size_t>(it.key0) * p.max_blocks + at];
        }
        return pg;  // not looked at here: the load goes on behind the tile before
      };
      auto load_tile = [&](const SeqItem& it, int j, int pg, uint8_t* dst, uint64_t* bar) {
        if constexpr (!PAGED) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::TILE);
            for (int c = 0; c < C::KCH; ++c)
              tma_load_3d_hint(dst + c * C::CHUNK, map, bar, c * 64, it.key0 + j * 128, it.kvh, keep);
          }
        } else {
          int a, e;
          tile_keys(it, j, a, e);
          const int i0 = a >> bsh, n = ((e + (1 << bsh) - 1) >> bsh) - i0;
          const int row = p.tiles_block <= 1 ? 0 : j % p.tiles_block * 128;
          if (lane == 0) mbar_arrive_expect_tx(bar, (n << bsh) * 128 * C::KCH);
          if (pg < 0 || pg >= p.num_blocks) {
            atomicCAS(p.status, 0u, kStatusInvalid | (kPSiteBlock << 8));
            pg = p.num_blocks;  // outside the map: reads as zeros
          }
          __syncwarp();
          const bool leader = elect_one();
          // Four to a turn, without a remainder of its own (it was half of this code).
#pragma unroll 1
          for (int i = i0; i < i0 + n; i += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int page = __shfl_sync(0xffffffffu, pg, i + k);
              if (leader && i + k < i0 + n) {
#pragma unroll
                for (int c = 0; c < C::KCH; ++c)
                  tma_load_4d(dst + c * C::CHUNK + ((i + k) << bsh) * 128, map, bar, c * 64, row, it.kvh, page);
              }
            }
          }
        }
      };
      auto zero_rows = [&]() -> bool {
        if (!wait_all(&v_raw[fix], raw_par >> fix & 1)) return false;
        raw_par ^= 1u << fix;
        uint8_t* v = sV + fix * C::TILE + (lane & 7) * 16;
#pragma unroll 1
        for (int r = lane >> 3; r < 128; r += 4)
          if (r < fix_a || r >= fix_e)
#pragma unroll
            for (int c = 0; c < C::KCH; ++c)
              *reinterpret_cast<uint4*>(v + c * C::CHUNK + r * 128) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[fix]);
        fix = -1;
        return true;
      };
      for (int ii = 0; ok; ++ii) {
        if (!(ok = wait_all(&item_full[ii % NI], (ii / NI) & 1))) break;
        const SeqItem it = items[ii % NI];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[ii % NI]);
        if (!it.valid) break;
        if (it.n == 0) continue;
        int pg = 0;
        if constexpr (PAGED) pg = pages_of(it, it.j0);
#pragma unroll 1
        for (int jj = 0; jj < it.n && ok; ++jj) {
          const int j = it.j0 + jj;
          // Q: tile 0 ahead of the item's first K tile, tile 1 behind it.
          auto load_q = [&](int t) -> bool {
            const int s = qc % C::QS;
            if (qc >= C::QS && !wait_all(&q_empty[s], ((qc / C::QS) - 1) & 1)) return false;
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full[s], C::KCH * 128 * p.G * p.tpt);
              for (int c = 0; c < C::KCH; ++c)
                tma_load_3d(sQ + s * C::QTILE + c * C::QCHUNK, &tmQ, &q_full[s], c * 64, it.kvh * p.G,
                            it.row0 + t * p.tpt);
            }
            ++qc;
            return true;
          };
          if (!is_v && jj == 0 && it.hi[0] > 0 && !(ok = load_q(0))) break;
          int pg_next = 0;
          if constexpr (PAGED) {
            if (jj + 1 < it.n) pg_next = pages_of(it, j + 1);
          }
          int a, e;
          tile_keys(it, j, a, e);
          const bool part = is_v && (a > 0 || e < 128);
          // A tile to be zeroed waits until the next load is out, or has no slot yet.
          bool loaded = false;
#pragma unroll 1
          for (;;) {
            if (!loaded && !(fix >= 0 && (part || (round && !__all_sync(0xffffffffu, mbar_test(&empty[slot], turn ^ 1)))))) {
              if (round && !(ok = wait_all(&empty[slot], turn ^ 1))) break;
              if (!skip) load_tile(it, j, pg, ring + slot * C::TILE, part ? &v_raw[slot] : &full[slot]);
              skip = false;
              loaded = true;
            }
            if (fix >= 0 && !(ok = zero_rows())) break;
            if (loaded) break;
          }
          if (!ok) break;
          if (part) fix = slot, fix_a = a, fix_e = e;
          if (++slot == slots) slot = 0, turn ^= 1, round = true;
          if (QT == 2 && !is_v && jj == 0 && it.hi[1] > 0) ok = load_q(1);
          pg = pg_next;
        }
      }
      if (ok && fix >= 0) ok = zero_rows();
      if (lane == 0) {
        // Every copy that was issued lands before the CTA leaves, on a timeout too.
        volatile int no_abort = 0;
        WaitCtl dw{p.status, &no_abort, 100000000ull};
#pragma unroll 1
        for (int i = max(0, qc - C::QS); i < qc; ++i)
          mbar_wait_far(&q_full[i % C::QS], (i / C::QS) & 1, dw, kQSiteDrain);
        if (fix >= 0) mbar_wait_far(&v_raw[fix], raw_par >> fix & 1, dw, kQSiteDrain);
#pragma unroll 1
        for (int i = 0; i < slots; ++i) {
          // Slots before `slot` were last loaded in this turn, the others in the one before.
          const bool now = i < slot;
          if ((!now && !round) || i == fix || (p.fault == 1 && !is_v && !round && i == 0)) continue;
          mbar_wait_far(&full[i], now ? turn : turn ^ 1, dw, kQSiteDrain);
        }
      }
      __syncwarp();
    } else if constexpr (NQ > 0) {
      // ---------------------------------------------------------------- issuers, few rows
      // S^T = K Q^T (128 keys x NQ rows) and O^T += V^T P^T (head columns x NQ rows); step c is
      // warpgroup c & 1's, with an accumulator of its own.  The issuing itself bounds a step on
      // 64-column heads (some 1700 cycles for both products from one thread, of which the tensor
      // pipe works 780), so the products have a warp each: warp 9 issues S, and finds the
      // items, which it has to know first; warp 10 issues P V.  S block and K slot c % KS share
      // s_full, V slot e % VS has o_done where VS is even (a slot's products are then always the
      // same warpgroup's).
      constexpr uint32_t id_s = idesc_f16(128, NQ, BF16, false, false);
      constexpr uint32_t id_o = idesc_f16(128, NQ, BF16, true, false);
      const bool leader = elect_one();  // the warp waits together, one thread issues
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, site)) != 0;
      };
      bool ok = true;
      int slot = 0;
      uint32_t par = 0;  // parity of the turn around the ring
      if (warp == 9) {
        const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dK = sdesc_sw128(smem_u32(sK), 16, 1024);
        ShareWalk<QT, kItemUnits> walk;
        walk.start(p, held, lane);
        SeqItem it{};
        int out = 0, in = 0, c = 0;  // items handed out, and begun here; steps issued
        bool have = false, next = true, ended = false;  // `it` is to be handed out; is to be found
        for (;;) {
          // Items go out as ring slots come free; waited for only when there is none to begin.
          while (ok && !ended) {
            if (next) have = walk.next(p, lane, it), next = false;
            const int s = out % NI;
            if (out >= NI) {
              const uint32_t turn = ((out / NI) - 1) & 1;
              if (out > in && !__all_sync(0xffffffffu, mbar_test(&item_empty[s], turn))) break;
              if (!(ok = wait(&item_empty[s], turn, kQSiteItemEmpty))) break;
            }
            if (!have) it.valid = 0, ended = true;
            if (leader) {
              items[s] = it;
              mbar_arrive(&item_full[s]);
            }
            __syncwarp();
            ++out;
            next = have;
          }
          if (!ok) break;
          // The next item is begun.  (Its slot was written by this warp.)
          const int s = in % NI;
          const int n = __shfl_sync(0xffffffffu, items[s].valid ? items[s].n : 0, 0);
          __syncwarp();
          if (leader) mbar_arrive(&item_empty[s]);
          if (n == 0) break;  // the end
          if (!(ok = wait(&q_full[in & 1], (in >> 1) & 1, kQSiteMmaQ))) break;
          const uint64_t q = sdesc_add(dQ, (in & 1) * C::QTILE);
          for (int i = 0; i < n; ++i, ++c) {
            ok = wait(&k_full[slot], par, kQSiteMmaK) && (c < C::KS || wait(&s_free[slot], par ^ 1, kQSiteMmaP));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              const uint64_t da = sdesc_add(dK, slot * C::TILE);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_ss(tbase + slot * NQ, sdesc_add(da, (kk >> 2) * C::CHUNK + (kk & 3) * 32),
                        sdesc_add(q, (kk >> 2) * C::QCHUNK + (kk & 3) * 32), id_s, kk > 0);
              umma_commit(&s_full[slot]);
              if (i + 1 == n) umma_commit(&q_empty[in & 1]);
            }
            if (++slot == C::KS) slot = 0, par ^= 1;
          }
          if (!ok) break;
          ++in;
        }
      } else {
        const uint64_t dV = sdesc_sw128(smem_u32(sV), C::CHUNK, 1024), dP = sdesc_sw128(smem_u32(sP), 16, 1024);
        int e = 0, oc0 = 0, oc1 = 0;  // steps issued; items begun per accumulator
        for (int ii = 0; ok; ++ii) {
          if (!(ok = wait(&item_full[ii % NI], (ii / NI) & 1, kQSiteItem))) break;
          const int n = __shfl_sync(0xffffffffu, items[ii % NI].valid ? items[ii % NI].n : 0, 0);
          __syncwarp();
          if (leader) mbar_arrive(&item_empty[ii % NI]);
          if (n == 0) break;
          for (int i = 0; i < n; ++i, ++e) {
            const int w = e & 1, pb = w * 2 + (e >> 1) % C::PB;
            ok = wait(&v_full[slot], par, kQSiteMmaV) && wait(&p_ready[pb], ((e >> 1) / C::PB) & 1, kQSiteMmaP);
            if (ok && i < 2) {
              // The first product of an accumulator overwrites it: read out by then.
              int& oc = w ? oc1 : oc0;
              if (oc > 0) ok = wait(&o_free[w], (oc - 1) & 1, kQSiteMmaO);
              ++oc;
            }
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              const uint64_t da = sdesc_add(dV, slot * C::TILE);
              const uint64_t db = sdesc_add(dP, (w * C::PB + (e >> 1) % C::PB) * C::PBUF);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_ss(tbase + C::O_COL(w), sdesc_add(da, kk * 2048),
                        sdesc_add(db, (kk >> 2) * (NQ * 128) + (kk & 3) * 32), id_o, (kk > 0 || i >= 2) ? 1u : 0u);
              umma_commit(&o_done[C::SHARE_V ? slot : w]);
              if (!C::SHARE_V) umma_commit(&v_empty[slot]);
            }
            if (++slot == C::VS) slot = 0, par ^= 1;
          }
        }
      }
      // Every product issued completes before tensor memory is released.
      uint64_t* end = warp == 9 ? &drain : &drain_pv;
      if (leader) umma_commit(end);
      volatile int no_abort = 0;
      WaitCtl dw{p.status, &no_abort, p.wait_ns};
      mbar_wait(end, 0, dw, kQSiteMmaDrain);
    } else if (lane == 0) {
      // ---------------------------------------------------------------- MMA issuer (warp 9)
      // One loop over the key tiles of all items.  Step j issues P V of its own tile and S of
      // the step after it, which may be the next item's first; the loop begins with a step
      // that has no P V.  (One thread feeds the tensor pipe: a body with every product once
      // keeps it in the instruction cache and its state in registers.)
      constexpr uint32_t id_qk = idesc_f16(128, 128, BF16, false, false);
      constexpr uint32_t id_pv = idesc_f16(128, D, BF16, false, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dK = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sV), C::CHUNK, 1024);
      int ii = 0, qc = 0, kc = 0, vc = 0;
      int sc0 = 0, sc1 = 0;  // score products issued per tile
      int ic0 = 0, ic1 = 0;  // items begun per tile
      int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0, q0 = 0, q1 = 0;  // the item: key tiles and Q loads
      int j = -1, jend = 0;
      bool ok = true;
      while (ok) {
        const bool real = j >= 0, last = j + 1 == jend;
        const int vs = vc % C::VS, ks = kc % C::KS;
        bool k_ok = false, v_ok = false, more = true;
        const SeqItem* nx = nullptr;
        // The next item that has key tiles; more: there is one.
        auto fetch = [&]() {
          for (;; ++ii) {
            nx = &items[ii % NI];
            if (!mbar_wait(&item_full[ii % NI], (ii / NI) & 1, wc, kQSiteItem)) { ok = false; return; }
            more = nx->valid != 0;
            if (!more || nx->n > 0) return;
            mbar_arrive(&item_empty[ii % NI]);
          }
        };
        // S of tile t for the step after this one.
        auto next_s = [&](int t, int lo, int hi, int q, int& sc) {
          bool go, need_q, fin;
          if (!last) {
            go = j + 1 >= lo && j + 1 < hi;
            need_q = j + 1 == lo;
            fin = j + 2 == hi;
          } else {
            if (!more) return;
            const int nlo = nx->lo[t], nhi = nx->hi[t];
            go = nhi > 0 && nlo == nx->j0;
            need_q = true;
            fin = nhi == nlo + 1;
            q = qc + (t == 1 && nx->hi[0] > 0 ? 1 : 0);
          }
          if (!go) return;
          const int qs = q % C::QS;
          if (need_q) ok = mbar_wait(&q_full[qs], (q / C::QS) & 1, wc, kQSiteMmaQ);
          if (ok && !k_ok) ok = mbar_wait(&k_full[ks], (kc / C::KS) & 1, wc, kQSiteMmaK);
          // The S block holds the step before's scores until they have been read.
          if (ok && C::SEP && sc > 0) ok = mbar_wait(&s_free[t], (sc - 1) & 1, wc, kQSiteMmaP);
          if (!ok) return;
          k_ok = true;
          tc_fence_after();
          const int b = QT == 2 ? t : (sc & 1);
          const uint64_t da = sdesc_add(dQ, qs * C::QTILE), db = sdesc_add(dK, ks * C::TILE);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
            umma_ss(tbase + b * 128, sdesc_add(da, off), sdesc_add(db, off), id_qk, kk > 0);
          }
          umma_commit(&s_full[b]);
          if (fin) umma_commit(&q_empty[qs]);
          ++sc;
        };
        // O_t += P V; pc: number of the step's scores.
        auto pv = [&](int t, int lo, int hi, int pc, int& ic) {
          if (j < lo || j >= hi) return;
          if (!v_ok) ok = mbar_wait(&v_full[vs], (vc / C::VS) & 1, wc, kQSiteMmaV);
          if (!ok) return;
          v_ok = true;
          // An item's first product overwrites the accumulator: read out by then.
          if (j == lo) {
            if (ic > 0) ok = mbar_wait(&o_free[t], (ic - 1) & 1, wc, kQSiteMmaO);
            ++ic;
          }
          const int pb = QT == 2 ? t : (pc & 1);
          if (ok) ok = mbar_wait(&p_ready[pb], (QT == 2 ? pc : pc >> 1) & 1, wc, kQSiteMmaP);
          if (!ok) return;
          tc_fence_after();
          const uint64_t db = sdesc_add(dV, vs * C::TILE);
          const uint32_t at = tbase + (C::SEP ? C::P_COL(t) : pb * 128u);
          const uint32_t acc = j > lo ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tbase + C::O_COL(t), at + kk * 8, sdesc_add(db, kk * 2048), id_pv, kk > 0 ? 1u : acc);
          umma_commit(&o_done[t]);
        };
        auto k_done = [&]() {  // a slot is only released once its load has landed
          if (last && !more) return;
          if (QT == 2 && !k_ok) ok = mbar_wait(&k_full[ks], (kc / C::KS) & 1, wc, kQSiteMmaK);
          if (!ok) return;
          umma_commit(&k_empty[ks]);
          ++kc;
        };
        const int p0 = sc0 - 1, p1 = sc1 - 1;
        if constexpr (QT == 1) {
          // S of the next step goes ahead of this step's P: two S blocks in turn.
          if (last) fetch();
          if (ok) next_s(0, lo0, hi0, q0, sc0);
          if (ok) k_done();
          if (ok) pv(0, lo0, hi0, p0, ic0);
        } else if constexpr (C::SEP) {
          if (last) fetch();
          if (ok) next_s(0, lo0, hi0, q0, sc0);
          if (ok) next_s(1, lo1, hi1, q1, sc1);
          if (ok) pv(0, lo0, hi0, p0, ic0);
          if (ok) pv(1, lo1, hi1, p1, ic1);
          if (ok) k_done();
        } else {
          pv(0, lo0, hi0, p0, ic0);
          if (ok && last) fetch();
          if (ok) next_s(0, lo0, hi0, q0, sc0);
          if (ok) pv(1, lo1, hi1, p1, ic1);
          if (ok) next_s(1, lo1, hi1, q1, sc1);
          if (ok) k_done();
        }
        if (!ok) break;
        if (real) {
          if (QT == 2 && !v_ok && !mbar_wait(&v_full[vs], (vc / C::VS) & 1, wc, kQSiteMmaV)) break;
          umma_commit(&v_empty[vs]);
          ++vc;
        }
        ++j;
        if (!last) continue;
        if (!more) break;
        lo0 = nx->lo[0], hi0 = nx->hi[0], lo1 = nx->lo[1], hi1 = nx->hi[1];
        j = nx->j0;
        jend = j + nx->n;
        if (hi0 > 0) q0 = qc++;
        if (QT == 2 && hi1 > 0) q1 = qc++;
        mbar_arrive(&item_empty[ii % NI]);
        ++ii;
      }
      // Every product issued completes before tensor memory is released.
      umma_commit(&drain);
      volatile int no_abort = 0;
      WaitCtl dw{p.status, &no_abort, p.wait_ns};
      mbar_wait(&drain, 0, dw, kQSiteMmaDrain);
    }
    __syncwarp();
  } else if constexpr (NQ > 0) {
    // ------------------------------------------------------------------ softmax, few rows
    // A decode step has G rows to an item.  With the rows along the 128 lanes of a score
    // tile, one warp of four would do all exponentials, 128 to a thread.  Here the keys lie
    // along the lanes: thread r holds the NQ scores of key r, and the two warpgroups take the
    // key tiles in turn, each with its own running maximum and accumulator; they are joined
    // at the item's end.  The maximum is shared by the warpgroup and stale as in the other
    // form: an exchange only when some score is more than 2^8 above it.
    regs_inc<C::SOFT_REGS>();
    constexpr int N = NQ;
    const int w = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;  // key of the tile; head column of the output
    const uint32_t lb = static_cast<uint32_t>(wq * 32);
    const uint32_t wg_bar = 1 + w;
    const int G = p.G;
    const float sl2 = p.scale_log2;
    uint8_t* myP = sP + w * C::PB * C::PBUF;
    int c = 0, pc = 0;  // steps before this item; steps of this warpgroup
    // Product k of this warpgroup.  (Its barrier's next phase is this warpgroup's too, VS being
    // even, and needs a P that is not written yet: no wait is more than one phase behind.)
    auto product = [&](int k) {  // step 2 k + w of all
      if (!C::SHARE_V) return mbar_wait(&o_done[w], k & 1, wc, kQSiteSoftO);
      return mbar_wait(&o_done[(2 * k + w) % C::VS], ((2 * k + w) / C::VS) & 1, wc, kQSiteSoftO);
    };
    for (int ii = 0;; ++ii) {
      // Waits end in a vote of all that share a named barrier, which has no time limit.
      if (!named_bar_and(3, 256, mbar_wait(&item_full[ii % NI], (ii / NI) & 1, wc, kQSiteItem))) break;
      const SeqItem& it = items[ii % NI];  // held until the item is done
      if (!it.valid) break;
      const int steps = it.n, rows = it.n_tok * G, pos = it.pos, nk = it.nk, j0 = it.j0;
      const int row0 = it.row0, kvh = it.kvh, part = it.part;
      // Keys up to sure_hi and from sure_lo on are seen by every row.
      const int sure_hi = p.causal ? min(pos, nk - 1) : nk - 1;
      const int sure_lo = p.window > 0 ? pos + it.n_tok - p.window : 0;
      float m[N], l[N], lr[N];
#pragma unroll
      for (int n = 0; n < N; ++n) m[n] = -INFINITY, l[n] = 0.f, lr[n] = 0.f;
      bool ok = true;
      const int s0 = (c & 1) == w ? 0 : 1;
      for (int s = s0; s < steps; s += 2) {
        const int b = (c + s) % C::KS;
        // This step's scores, and P's buffer free of the product that read it last.
        bool got = mbar_wait(&s_full[b], ((c + s) / C::KS) & 1, wc, kQSiteSoftS);
        if (got && pc >= C::PB) got = product(pc - C::PB);
        got = __all_sync(0xffffffffu, got);
        uint32_t sr[N];
        if (got) {
          tc_fence_after();
          tmem_ld16(tmem_addr(tbase, lb, b * N), sr);
          tmem_wait_ld();
          reg_fence(sr);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[b]);
        }
        const int kc0 = (j0 + s) * 128, key = kc0 + r;
        const bool masked = kc0 + 127 > sure_hi || kc0 < sure_lo;
        float x[N];
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = n < rows ? __uint_as_float(sr[n]) * sl2 : -INFINITY;
        if (masked) {
          int tok = 0, g = 0;
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const int kl = p.causal ? min(pos + tok, nk - 1) : nk - 1;
            if (key > kl || (p.window > 0 && key <= pos + tok - p.window)) x[n] = -INFINITY;
            if (++g == G) g = 0, ++tok;
          }
        }
        bool need = s == s0;
        float wm[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
          wm[n] = -INFINITY;
          if (n < rows) wm[n] = warp_max(x[n]);
          need |= wm[n] - m[n] > 8.0f;
        }
        // One vote a step: no exchange, and nobody's wait ran out.
        if (!named_bar_and(wg_bar, 128, got && !need)) {
          // The accumulator's last product is done before it is rescaled (and P's other buffer,
          // which takes the maxima, free).
          if (got && pc > 0) got = product(pc - 1);
          ok = named_bar_and(wg_bar, 128, got);
          if (!ok) break;
          tc_fence_after();
          float* ex = reinterpret_cast<float*>(myP + pc % C::PB * C::PBUF);  // [4][N]
          if (lane < N) {
            float mine = wm[0];
#pragma unroll
            for (int n = 1; n < N; ++n) mine = lane == n ? wm[n] : mine;
            ex[wq * N + lane] = mine;
          }
          named_bar_sync(wg_bar, 128);
          float f[N];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const float t = fmaxf(fmaxf(ex[n], ex[N + n]), fmaxf(ex[2 * N + n], ex[3 * N + n]));
            const float mn = fmaxf(m[n], t);
            f[n] = mn - m[n] > 0.f ? ex2_approx(m[n] - mn) : 1.0f;
            m[n] = mn;
            l[n] *= f[n];
            lr[n] *= f[n];
          }
          if (s != s0) {
            uint32_t o[N];
            tmem_ld16(tmem_addr(tbase, lb, C::O_COL(w)), o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int n = 0; n < N; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n]);
            tmem_st16(tmem_addr(tbase, lb, C::O_COL(w)), o);
            tmem_wait_st();
            tc_fence_before();
          }
          named_bar_sync(wg_bar, 128);  // every warp has read the maxima: P may go over them
        }
        // P^T, K-major rows of 64 keys with 128-byte swizzle: 16-byte unit u of row n at u ^ (n % 8).
        uint8_t* dst = myP + pc % C::PB * C::PBUF + (r >> 6) * (N * 128) + (r & 7) * 2;
        const int u = (r & 63) >> 3;
#pragma unroll
        for (int n = 0; n < N; n += 2) {
          if (n >= rows) continue;  // columns of no row: nothing reads their output
          const float e0 = ex2_approx(x[n] - (m[n] == -INFINITY ? 0.f : m[n]));
          const float e1 = ex2_approx(x[n + 1] - (m[n + 1] == -INFINITY ? 0.f : m[n + 1]));
          const uint32_t pk = pack2<BF16>(e0, e1);
          float r0, r1;
          unpack2<BF16>(pk, r0, r1);
          l[n] += e0;
          l[n + 1] += e1;
          lr[n] += r0;
          lr[n + 1] += r1;
          *reinterpret_cast<uint16_t*>(dst + n * 128 + ((u ^ (n & 7)) << 4)) = static_cast<uint16_t>(pk);
          *reinterpret_cast<uint16_t*>(dst + (n + 1) * 128 + ((u ^ ((n + 1) & 7)) << 4)) = static_cast<uint16_t>(pk >> 16);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[w * 2 + pc % C::PB]);
        ++pc;
      }
      // The item's end: the sums over the keys, then both warpgroups' parts joined.
      const bool mine = steps > s0;  // this warpgroup had steps
      if (ok && mine) ok = product(pc - 1);
      float* ex = reinterpret_cast<float*>(myP);  // [4][2][N] sums, [N] maxima (P is not read any more)
      if (steps > 0) {
        // Each exchange halves the rows that a lane sums: 31 instead of 160 for all, and a
        // quarter of the code.  Lane 2 n (and 2 n + 1) ends up with the warp's sums of row n.
        static_assert(N == 16, "four halvings");
#pragma unroll
        for (int h = N / 2; h >= 1; h >>= 1) {
          const bool up = lane & (2 * h);
#pragma unroll
          for (int n = 0; n < h; ++n) {
            const float a = up ? l[n] : l[n + h], q = up ? lr[n] : lr[n + h];
            l[n] = (up ? l[n + h] : l[n]) + __shfl_xor_sync(0xffffffffu, a, 2 * h);
            lr[n] = (up ? lr[n + h] : lr[n]) + __shfl_xor_sync(0xffffffffu, q, 2 * h);
            m[n] = up ? m[n + h] : m[n];
          }
        }
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
        lr[0] += __shfl_xor_sync(0xffffffffu, lr[0], 1);
        // (P's buffer is free once this warpgroup's last product is done, for all its warps.)
        ok = named_bar_and(wg_bar, 128, ok);
        if (ok && !(lane & 1)) {
          ex[(wq * 2) * N + (lane >> 1)] = l[0];
          ex[(wq * 2 + 1) * N + (lane >> 1)] = lr[0];
          if (wq == 0) ex[8 * N + (lane >> 1)] = m[0];
        }
        tc_fence_before();
      }
      if (!named_bar_and(3, 256, ok)) break;
      tc_fence_after();
      constexpr int H2 = N / 2;  // rows of this warpgroup's half
      const float* e0 = reinterpret_cast<const float*>(sP);
      const float* e1 = reinterpret_cast<const float*>(sP + C::PB * C::PBUF);
      const int n0 = w * H2;
      if (n0 < rows) {
        // Which warpgroups have a part: with one step only the one whose turn it was.
        const bool has0 = steps > 1 || (steps == 1 && (c & 1) == 0), has1 = steps > 1 || (steps == 1 && (c & 1) == 1);
        int tok = n0 / G, g = n0 - tok * G;
        // Row by row: unrolled, this was 24 KB of code, run cold at every item's end.
#pragma unroll 1
        for (int n = n0; n < min(rows, n0 + H2); ++n) {
          {
            uint32_t o0[1], o1[1];
            tmem_ld1(tmem_addr(tbase, lb, C::O_COL(0) + n), o0);
            tmem_ld1(tmem_addr(tbase, lb, C::O_COL(1) + n), o1);
            tmem_wait_ld();
            reg_fence(o0);
            reg_fence(o1);
            // A part counts if its sum is not exactly zero, which means a row that sees none of its
            // keys.  The maxima pass over a NaN (and are -inf where every score is one); the sums
            // carry it, and the weights of +inf, NaN too, through to O and LSE.
            float l0 = 0.f, r0 = 0.f, l1 = 0.f, r1 = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (has0) l0 += e0[q * 2 * N + n], r0 += e0[(q * 2 + 1) * N + n];
              if (has1) l1 += e1[q * 2 * N + n], r1 += e1[(q * 2 + 1) * N + n];
            }
            const float m0 = l0 != 0.f ? e0[8 * N + n] : -INFINITY, m1 = l1 != 0.f ? e1[8 * N + n] : -INFINITY;
            const float M = fmaxf(m0, m1);
            float L = 0.f, R = 0.f, y = 0.f;
            if (l0 != 0.f) {
              const float a = ex2_approx(m0 - M);
              L = a * l0, R = a * r0, y = a * __uint_as_float(o0[0]);
            }
            if (l1 != 0.f) {
              const float a = ex2_approx(m1 - M);
              L += a * l1, R += a * r1, y += a * __uint_as_float(o1[0]);
            }
            const float lse = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
            y *= L == 0.f ? 0.f : 1.0f / R;
            const int row = row0 + tok, head = kvh * G + g;
            if (part < 0) {
              if (r < p.d)
                p.O[row * p.o_row + head * p.o_head + r] = static_cast<uint16_t>(pack2<BF16>(y, 0.f));
              if (r == 0) p.LSE[static_cast<size_t>(head) * p.T + row] = lse;
            } else {
              const size_t prow = static_cast<size_t>(part) * 128 + n;
              if (r < D) p.O_part[prow * D + r] = y;
              if (r == 0) p.LSE_part[prow] = lse;
            }
          }
          if (++g == G) g = 0, ++tok;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (steps > 0) {
          // An accumulator without steps in this item is not waited for.
          if (steps > 1 || (c & 1) == 0) mbar_arrive(&o_free[0]);
          if (steps > 1 || (c & 1) == 1) mbar_arrive(&o_free[1]);
        }
        mbar_arrive(&item_empty[ii % NI]);
      }
      c += steps;
    }
  } else {
    // ------------------------------------------------------------------ softmax
    regs_inc<C::SOFT_REGS>();
    const int t = warp >> 2, wq = warp & 3;
    const int r_loc = wq * 32 + lane;
    const int G = p.G, tpt = p.tpt;
    const int tok_r = r_loc / G, g_r = r_loc - tok_r * G;
    const uint32_t o_col = C::O_COL(t);
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32);
    const float sl2 = p.scale_log2;
    int sc = 0;  // steps of this tile so far
    bool ok = t < QT;
    for (int ii = 0; ok; ++ii) {
      ok = __all_sync(0xffffffffu, mbar_wait(&item_full[ii % NI], (ii / NI) & 1, wc, kQSiteItem));
      if (!ok) break;
      const SeqItem& it = items[ii % NI];  // held until the item is done
      if (!it.valid) break;
      const int lo = t ? it.lo[1] : it.lo[0], steps = (t ? it.hi[1] : it.hi[0]) - lo;
      const int tok = t * tpt + tok_r;
      const bool row_ok = tok_r < tpt && tok < it.n_tok;
      const bool live = __any_sync(0xffffffffu, row_ok);
      const int pos = it.pos + tok;
      const int klast = p.causal ? min(pos, it.nk - 1) : it.nk - 1;
      const int kfirst = p.window > 0 ? pos - p.window + 1 : 0;
      float m = -INFINITY;  // running maximum, log2 units
      float l = 0.f;        // sum of the weights: the log-sum-exp
      float lr = 0.f;       // sum of the weights as rounded for P V: the divisor of O
      for (int step = 0; step < steps; ++step, ++sc) {
        // QT = 1: the two S blocks in turn; else one block to a tile.
        const int buf = QT == 1 ? (sc & 1) : t;
        const uint32_t par = QT == 1 ? ((sc >> 1) & 1) : (sc & 1);
        const uint32_t s_col = buf * 128u;
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[buf], par, wc, kQSiteSoftS));
        if (!ok) break;
        if (live) {
          tc_fence_after();
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tmem_ld32(tmem_addr(tbase, lane_base, s_col + 32 * c), *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
          tmem_wait_ld();
          reg_fence(sr);
          if (C::SEP) {  // the S block may take the next scores
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[t]);
          }
          // Keys past the row's last one or before its window.
          const int kc0 = (lo + step) * 128;
          const int hi_lim = klast - kc0 + 1, lo_lim = kfirst - kc0;
          if (__any_sync(0xffffffffu, hi_lim < 128 || lo_lim > 0)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // Bits lo .. hi - 1 of 32 keys: two comparisons a key were 5 KB more of code.
              const int hi = min(max(hi_lim - 32 * c, 0), 32), lo = min(max(lo_lim - 32 * c, 0), 32);
              const uint32_t keep = static_cast<uint32_t>(((1ull << hi) - 1) & ~((1ull << lo) - 1));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(keep & (1u << i))) sr[32 * c + i] = __float_as_uint(-INFINITY);
            }
          }
          float mx[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx[k] = fmax3(__uint_as_float(sr[k]), __uint_as_float(sr[k + 8]), __uint_as_float(sr[k + 16]));
#pragma unroll
          for (int i = 24; i < 120; i += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mx[k] = fmax3(mx[k], __uint_as_float(sr[i + k]), __uint_as_float(sr[i + k + 8]));
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(sr[120 + k]));
          mx[0] = fmax3(mx[0], mx[1], mx[2]);
          mx[3] = fmax3(mx[3], mx[4], mx[5]);
          mx[6] = fmaxf(mx[6], mx[7]);
          mx[0] = fmax3(mx[0], mx[3], mx[6]);
          const float m_new = fmaxf(m, mx[0] * sl2);
          if (step == 0) {
            m = m_new;
          } else {
            // The stale maximum is kept until it is more than 2^8 behind.
            const bool need = m_new - m > 8.0f;
            if (__any_sync(0xffffffffu, need)) {
              const float f = need ? ex2_approx(m - m_new) : 1.0f;
              if (need) m = m_new;
              l *= f;
              lr *= f;
              ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (sc - 1) & 1, wc, kQSiteSoftO));
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                tmem_ld32(tmem_addr(tbase, lane_base, o_col + 32 * c), r);
                tmem_wait_ld();
                reg_fence(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                tmem_st32(tmem_addr(tbase, lane_base, o_col + 32 * c), r);
              }
            }
          }
          const uint64_t sl2x2 = f2_pack(sl2, sl2);
          const float neg_m = (m == -INFINITY) ? 0.f : -m;
          const uint64_t negm2 = f2_pack(neg_m, neg_m);
          uint64_t sum2[4] = {0, 0, 0, 0}, sumr2[4] = {0, 0, 0, 0};
          if (C::SEP && step > 0) {  // the P V product before may still read P
            ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (sc - 1) & 1, wc, kQSiteSoftO));
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t p_col = C::SEP ? C::P_COL(t) : s_col;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int k = 64 * h + 2 * i;
              float a, b;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), sl2x2, negm2), a, b);
              a = ex2_approx(a);
              b = ex2_approx(b);
              sum2[i & 3] = f2_add(sum2[i & 3], f2_pack(a, b));
              pk[i] = pack2<BF16>(a, b);
              float r0, r1;
              unpack2<BF16>(pk[i], r0, r1);
              sumr2[i & 3] = f2_add(sumr2[i & 3], f2_pack(r0, r1));
            }
            tmem_st32(tmem_addr(tbase, lane_base, p_col + 32 * h), pk);
          }
          float x0, x1;
          f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), x0, x1);
          l += x0 + x1;
          f2_unpack(f2_add(f2_add(sumr2[0], sumr2[1]), f2_add(sumr2[2], sumr2[3])), x0, x1);
          lr += x0 + x1;
          tmem_wait_st();
          tc_fence_before();
        } else if (C::SEP) {
          // A warp without rows keeps the barriers' counts.
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[t]);
          if (step > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (sc - 1) & 1, wc, kQSiteSoftO));
            if (!ok) break;
          }
        }
        // QT = 1: S of the item's last step was issued ahead of the P V before it, which may
        // be pending.  It is waited for before the last P is handed over, so that no later
        // product can complete meanwhile and the wait below stays within one phase.
        if (QT == 1 && step == steps - 1 && step >= 1) {
          ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (sc - 1) & 1, wc, kQSiteSoftO));
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[buf]);
      }
      if (!ok) break;
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (sc - 1) & 1, wc, kQSiteSoftO));
        if (!ok) break;
        tc_fence_after();
      }
      // A row that sees no key: O = 0, LSE = -inf.  Its sum is exactly zero (any other has weights of
      // about one and more); the sum of a row that sees a NaN or a score of +inf is NaN, and so are
      // its O and LSE.
      const float inv_l = l == 0.f ? 0.f : 1.0f / lr;
      const float lse = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
      const int part = PAGED ? it.part : -1;  // packed items are never cut
      if (live) {
        const int row = it.row0 + tok, head = it.kvh * G + g_r;
        uint16_t* orow = p.O + row * p.o_row + head * p.o_head;
        const size_t prow = (static_cast<size_t>(max(part, 0)) * QT + t) * 128 + r_loc;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          if (steps > 0) {
            tmem_ld32(tmem_addr(tbase, lane_base, o_col + 32 * c), r);
            tmem_wait_ld();
            reg_fence(r);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
          }
          if (part < 0) {
            if (row_ok) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (c * 32 + 8 * i < p.d) {
                  uint32_t w[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    w[e] = pack2<BF16>(__uint_as_float(r[8 * i + 2 * e]) * inv_l,
                                       __uint_as_float(r[8 * i + 2 * e + 1]) * inv_l);
                  *reinterpret_cast<uint4*>(orow + c * 32 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
          } else if (row_ok && l != 0.f) {
            float4* dst = reinterpret_cast<float4*>(p.O_part + prow * D + c * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(__uint_as_float(r[4 * i]) * inv_l, __uint_as_float(r[4 * i + 1]) * inv_l,
                                   __uint_as_float(r[4 * i + 2]) * inv_l, __uint_as_float(r[4 * i + 3]) * inv_l);
          }
        }
        if (row_ok) {
          if (part < 0) p.LSE[static_cast<size_t>(head) * p.T + row] = lse;
          else p.LSE_part[prow] = lse;
        }
      }
      if (steps > 0) tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (steps > 0) mbar_arrive(&o_free[t]);
        mbar_arrive(&item_empty[ii % NI]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ------------------------------------------------------------------------------------
// merge of the partials
// ------------------------------------------------------------------------------------

// CTA x merges the block of rows that starts in share x and goes on in the next ones, if
// there is one (blockIdx.y: every gridDim.y-th row; a warp to a row):
//   M = max L_s,  O = sum e^{L_s - M} O_s / sum e^{L_s - M},  LSE = M + ln sum e^{L_s - M}.
// The forward kernel left the block's place; finding it again from the lengths took longer
// than the merge.
template <int D, bool BF16, int QT>
__global__ void __launch_bounds__(256) fa2_seq_merge_kernel(const SeqParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x;
  griddep_wait();
  const int4 at = p.merge[c];
  const int parts = min(at.w, static_cast<int>(gridDim.x) - c);
  if (parts < 2) return;
  const int n_tok = min(min(at.y, QT * p.tpt), p.T - at.x);
  constexpr int PER = D / 32, U = 4;
  for (int i = blockIdx.y * 8 + warp; i < n_tok * p.G; i += 8 * gridDim.y) {
    const int tok = i / p.G, g = i - tok * p.G;
    const int t = QT == 1 ? 0 : tok / p.tpt;
    const int r = t * 128 + (tok - t * p.tpt) * p.G + g;
    const auto slot = [&](int s) {  // row of part s: the first is its share's second slot
      return (static_cast<size_t>(2 * (c + s) + (s == 0 ? 1 : 0)) * QT) * 128 + r;
    };
    // The maximum passes over a NaN; the weights then bring it into the sums.
    float M = -INFINITY;
    for (int s = lane; s < parts; s += 32) M = fmaxf(M, p.LSE_part[slot(s)]);
    M = warp_max(M);
    float acc[PER] = {}, wsum = 0.f;
    for (int s0 = 0; s0 < parts; s0 += U) {
      float L[U], v[U][PER];
#pragma unroll
      for (int k = 0; k < U; ++k) L[k] = s0 + k < parts ? p.LSE_part[slot(s0 + k)] : -INFINITY;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        // A part of whose keys the row sees none was not written.
        if (L[k] != -INFINITY) {
          const float* src = p.O_part + slot(s0 + k) * D + lane * PER;
#pragma unroll
          for (int e = 0; e < PER; e += 2) {
            const float2 f = *reinterpret_cast<const float2*>(src + e);
            v[k][e] = f.x;
            v[k][e + 1] = f.y;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (L[k] == -INFINITY) continue;
        const float w = exp2f((L[k] - M) * 1.4426950408889634f);
        wsum += w;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
      }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;  // 0: no part with a key
    const int row = at.x + tok, head = at.z * p.G + g;
    uint16_t* dst = p.O + row * p.o_row + head * p.o_head + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e += 2)
      if (lane * PER + e < p.d)
        *reinterpret_cast<uint32_t*>(dst + e) = pack2<BF16>(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0)
      p.LSE[static_cast<size_t>(head) * p.T + row] = wsum == 0.f ? -INFINITY : M + logf(wsum);
  }
}

}  // namespace fa2
