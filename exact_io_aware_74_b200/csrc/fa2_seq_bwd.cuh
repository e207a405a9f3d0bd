// Backward over packed sequences with grouped heads.
//
// The mathematics, the tiles and the tensor-memory plans are those of the dense default
// backward (fa2_bwd.cuh): per 128-key tile, S^T = K Q^T and dP^T = V dO^T, P^T from the
// saved log-sum-exp, dV += P^T dO, dS^T = P^T (dP^T - D), dK += dS^T Q, and dQ partials
// dS K added into a float accumulator by TMA.  What differs:
//
//   * A query tile holds the G heads of one key/value head (row = token * G + head,
//     128 / G tokens), so that dK and dV of a shared head sum over its query heads in
//     the accumulators, in a fixed order, and a short sequence fills few tiles.
//   * A work item is one (sequence, key/value head, 128-key tile).  The items are found
//     on the device from the lengths, most query tiles first, and handed out by cluster
//     launch control (see fa2_seq_fwd.cuh); no counter in memory.
//   * Per-row data of the workspace (D, LSE log2 e, the dQ accumulator) is laid out by
//     query tile: sequence b starts at tile cu[b] / (128 / G) + b, which leaves room for
//     its last, partial tile.
//   * Rows of K, V, Q and dO tiles that belong to no row of the sequence are zeroed in
//     shared memory by a warp of its own before any product reads them: a product with
//     a zero weight would still pass on a NaN of the neighbouring sequence.
//
// Where the items are too few for the SMs, the query tiles of each key tile are cut into
// `split` parts, one item each: dK and dV then go to the workspace as float parts, which
// the last kernel sums in order (repeatable all the same).
//
// Kernels per call, chained by programmatic dependent launch: fa2_seq_bwd_pre_kernel
// (D, LSE log2 e, zeroed accumulator), fa2_seq_bwd_kernel, fa2_seq_bwd_dq_kernel
// (dQ = scale * accumulator, to 16 bits and to its place; split dK and dV).
#pragma once

#include <cstdint>

#include "fa2_seq_fwd.cuh"
#include "ptx.cuh"

namespace fa2 {

struct SeqBwdParams {
  const uint16_t *O, *dO;
  uint16_t *dQ, *dK, *dV;
  long long o_row, o_head, do_row, do_head, dq_row, dq_head, dk_row, dk_head, dv_row, dv_head;
  const float* LSE;  // [H][T]
  float *Dg, *Lg;    // [Hkv][tiles * 128]
  float* acc;        // [Hkv][tiles * 128][D]
  float* kv_part;    // split > 1: [split][dV, dK][T][Hkv][D]
  const int* cu;
  unsigned int* status;
  unsigned long long wait_ns;
  int B, T, Hkv, G, d, tpt, tiles;  // tiles: query tiles of one key/value head, room included
  int causal, window, fault, head_group;
  int split;         // parts that a key tile's query tiles are cut into
  float scale, scale_log2;
};

// Query tiles [i0, i0 + n) that see key tile j of a sequence of len rows.
__device__ __forceinline__ void query_range(const SeqBwdParams& p, int len, int j, int& i0, int& n) {
  const int n_q = (len + p.tpt - 1) / p.tpt;
  i0 = p.causal ? j * 128 / p.tpt : 0;
  int e = n_q;
  if (p.window > 0) {
    const long long t = static_cast<long long>(j) * 128 + 127 + p.window - 1;  // last token that sees the tile
    e = static_cast<int>(min(static_cast<long long>(n_q), t / p.tpt + 1));
  }
  n = e - i0;
}

// First query tile of sequence b.
__device__ __forceinline__ int tile_base(const SeqBwdParams& p, int b) {
  return min(max(p.cu[b], 0), p.T) / p.tpt + b;
}

// The token and query head of row r (of tiles * 128), or false: the row is padding.
__device__ __forceinline__ bool row_of(const SeqBwdParams& p, int r, int& row, int& g) {
  const int tile = r >> 7, rl = r & 127, tok = rl / p.G;
  int i = 0, j = p.B;  // the last sequence that starts at or before the tile
  while (j - i > 1) {
    const int m = (i + j) >> 1;
    if (tile_base(p, m) <= tile) i = m; else j = m;
  }
  const int s = min(max(p.cu[i], 0), p.T), n = rows_of(p.cu, p.T, i);
  const int at = (tile - tile_base(p, i)) * p.tpt + tok;
  row = s + at;
  g = rl - tok * p.G;
  return tok < p.tpt && at >= 0 && at < n;
}

// ------------------------------------------------------------------------------------
// 1. preprocess
// ------------------------------------------------------------------------------------

template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa2_seq_bwd_pre_kernel(const SeqBwdParams p) {
  constexpr int TPR = D / 8, RPB = 256 / TPR;  // threads to a row, rows to a CTA
  griddep_launch_dependents();
  griddep_wait();
  const int sub = threadIdx.x % TPR;
  const int r = blockIdx.x * RPB + threadIdx.x / TPR, hk = blockIdx.y;
  const size_t at = static_cast<size_t>(hk) * p.tiles * 128 + r;
  int row, g;
  const bool ok = row_of(p, r, row, g);
  const int h = hk * p.G + g;
  float acc = 0.f;
  if (ok && sub * 8 < p.d) {
    const uint4 a = *reinterpret_cast<const uint4*>(p.O + row * p.o_row + h * p.o_head + sub * 8);
    const uint4 b = *reinterpret_cast<const uint4*>(p.dO + row * p.do_row + h * p.do_head + sub * 8);
    const uint32_t pa[4] = {a.x, a.y, a.z, a.w}, pb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a0, a1, b0, b1;
      unpack2<BF16>(pa[i], a0, a1);
      unpack2<BF16>(pb[i], b0, b1);
      acc = fmaf(a0, b0, acc);
      acc = fmaf(a1, b1, acc);
    }
  }
  float4* z = reinterpret_cast<float4*>(p.acc + at * D + sub * 8);
  z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
  z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int o = TPR / 2; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o, TPR);
  if (sub == 0) {
    p.Dg[at] = ok ? acc : 0.f;
    p.Lg[at] = ok ? p.LSE[static_cast<size_t>(h) * p.T + row] * 1.4426950408889634f : INFINITY;
  }
}

// ------------------------------------------------------------------------------------
// 3. dQ
// ------------------------------------------------------------------------------------

template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa2_seq_bwd_dq_kernel(const SeqBwdParams p) {
  constexpr int TPR = D / 8, RPB = 256 / TPR;
  griddep_wait();
  const int sub = threadIdx.x % TPR;
  const int r = blockIdx.x * RPB + threadIdx.x / TPR;
  if (static_cast<int>(blockIdx.y) >= p.Hkv) {
    // Split key tiles: dV and dK of packed row r, the parts summed in order.
    if (r >= p.T || sub * 8 >= p.d) return;
    const int hk = blockIdx.y - p.Hkv;
    int i = 0, j = p.B;  // the sequence of row r
    while (j - i > 1) {
      const int m = (i + j) >> 1;
      if (p.cu[m] <= r) i = m; else j = m;
    }
    const int key = r - min(max(p.cu[i], 0), p.T), len = rows_of(p.cu, p.T, i);
    if (key < 0 || key >= len) return;
    int i0, n;
    query_range(p, len, key >> 7, i0, n);
    const int parts = min(p.split, n);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float a[8] = {};
      for (int k = 0; k < parts; ++k) {
        const float4* s = reinterpret_cast<const float4*>(
            p.kv_part + (((static_cast<size_t>(k) * 2 + w) * p.T + r) * p.Hkv + hk) * D + sub * 8);
        const float4 x = s[0], y = s[1];
        a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
        a[4] += y.x, a[5] += y.y, a[6] += y.z, a[7] += y.w;
      }
      const float f = w ? p.scale : 1.0f;
      uint16_t* dst = w ? p.dK + r * p.dk_row + hk * p.dk_head : p.dV + r * p.dv_row + hk * p.dv_head;
      *reinterpret_cast<uint4*>(dst + sub * 8) =
          make_uint4(pack2<BF16>(a[0] * f, a[1] * f), pack2<BF16>(a[2] * f, a[3] * f), pack2<BF16>(a[4] * f, a[5] * f),
                     pack2<BF16>(a[6] * f, a[7] * f));
    }
    return;
  }
  const int hk = blockIdx.y;
  int row, g;
  if (!row_of(p, r, row, g) || sub * 8 >= p.d) return;
  const float4* s = reinterpret_cast<const float4*>(p.acc + (static_cast<size_t>(hk) * p.tiles * 128 + r) * D + sub * 8);
  const float4 a = s[0], b = s[1];
  const float f = p.scale;
  *reinterpret_cast<uint4*>(p.dQ + row * p.dq_row + (hk * p.G + g) * p.dq_head + sub * 8) =
      make_uint4(pack2<BF16>(a.x * f, a.y * f), pack2<BF16>(a.z * f, a.w * f), pack2<BF16>(b.x * f, b.y * f),
                 pack2<BF16>(b.z * f, b.w * f));
}

// ------------------------------------------------------------------------------------
// 2. main kernel
// ------------------------------------------------------------------------------------

struct SeqBwdItem {
  int row0, n;     // first packed row and length of the sequence
  int kvh, j;      // key/value head, key tile
  int i0, n_it;    // query tiles i0 .. i0 + n_it - 1
  int qt0, valid;  // the sequence's first query tile in the workspace
  int part, pad;   // SPLIT: which part of the key tile's query tiles
};

template <int D_>
struct SeqBwdCfg {
  static constexpr int D = D_;
  static_assert(D == 64 || D == 128, "tile widths");
  static constexpr int KCH = D / 64, CHUNK = 128 * 128, TILE = 128 * D * 2;
  static constexpr int ST = 2;                  // (Q, dO) ring stages
  static constexpr int KVB = D == 64 ? 2 : 1;   // K, V buffers
  static constexpr bool PIPE = D == 64;         // software-pipelined steps (tensor memory has room)
  static constexpr int DS_BYTES = 128 * 128 * 2, LD_BYTES = ST * 2 * 128 * 4, CTRL_BYTES = 1024;
  static constexpr int SMEM = (2 * KVB + 2 * ST) * TILE + DS_BYTES + LD_BYTES + CTRL_BYTES;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr int THREADS = 384;
  // Tensor memory: S^T [0,128), dP^T [128,256), dV, dK; dQ shares dP^T's columns at D = 128.
  static constexpr uint32_t C_S = 0, C_DP = 128, C_DV = 256, C_DK = 256 + D, C_DQ = D == 128 ? 128 : 384;
  __host__ __device__ static constexpr uint32_t C_P(int g) { return D == 64 ? 448u + 32u * g : 64u * g; }
  __host__ __device__ static constexpr uint32_t C_DS(int g) { return D == 128 ? 64u * g + 32u : C_DP + 64u * g; }
};

constexpr int kHeldBwd = 96;  // as kHeld; what shared memory has left at D = 128

struct SeqBwdCtrl {
  uint4 clc_response;
  SeqBwdItem items[kSeqItems];
  uint64_t item_full[kSeqItems], item_empty[kSeqItems], clc_full;
  uint64_t kv_full[2], kv_raw[2], kv_empty[2], acc_free;
  uint64_t qdo_full[2], qdo_raw[2], qdo_empty[2], q_full[2], q_raw[2], q_empty[2];
  uint64_t s_full, dp_full, p_ready, ds_ready, dq_full, dq_drained, drain, fin;
  uint32_t tmem_slot;
  int abort_flag;
  int held[kHeldBwd];  // the scheduling warp's
};

__device__ __forceinline__ void bulk_load(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(gmem_src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

enum SeqBwdSite : uint32_t {
  kRSiteAlign = 100, kRSiteItem, kRSiteItemEmpty, kRSiteClc, kRSiteProd, kRSiteFix, kRSiteMmaKV, kRSiteMmaQ,
  kRSiteMmaP, kRSiteMmaDS, kRSiteMmaDrained, kRSiteMmaAcc, kRSiteMmaDrain, kRSiteCmpQ, kRSiteCmpS, kRSiteCmpDP,
  kRSiteCmpDQ, kRSiteDrain
};

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(384, 1)
fa2_seq_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                   const __grid_constant__ CUtensorMap tmdQ, const SeqBwdParams p) {
  using C = SeqBwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0u, 4u | (kRSiteAlign << 8));
    return;
  }
  griddep_launch_dependents();
  uint8_t* sK = smem_raw;
  uint8_t* sV = sK + C::KVB * C::TILE;
  uint8_t* sQ = sV + C::KVB * C::TILE;
  uint8_t* sdO = sQ + C::ST * C::TILE;
  uint8_t* sDS = sdO + C::ST * C::TILE;  // dS^T, MN-major, for the dQ product; then dQ staging
  float* sLD = reinterpret_cast<float*>(sDS + C::DS_BYTES);  // [ST][2][128]: L, D
  SeqBwdCtrl& ctl = *reinterpret_cast<SeqBwdCtrl*>(sDS + C::DS_BYTES + C::LD_BYTES);
  static_assert(sizeof(SeqBwdCtrl) <= C::CTRL_BYTES, "control block too large");
  constexpr int NI = kSeqItems;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  WaitCtl wc{p.status, &ctl.abort_flag, p.wait_ns};

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int i = 0; i < NI; ++i) {
      mbar_init(&ctl.item_full[i], 1);
      mbar_init(&ctl.item_empty[i], 3 + 8);  // producer, MMA, fix, compute warps
    }
    mbar_init(&ctl.clc_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.kv_full[b], 1);
      mbar_init(&ctl.kv_raw[b], 1);
      mbar_init(&ctl.kv_empty[b], 1);
      mbar_init(&ctl.qdo_full[b], 1);
      mbar_init(&ctl.qdo_raw[b], 1);
      mbar_init(&ctl.qdo_empty[b], C::PIPE ? 1 : 2);
      mbar_init(&ctl.q_full[b], 1);
      mbar_init(&ctl.q_raw[b], 1);
      mbar_init(&ctl.q_empty[b], 1);
    }
    mbar_init(&ctl.acc_free, 8);
    mbar_init(&ctl.s_full, 1);
    mbar_init(&ctl.dp_full, 1);
    mbar_init(&ctl.p_ready, 8);
    mbar_init(&ctl.ds_ready, 8);
    mbar_init(&ctl.dq_full, 1);
    mbar_init(&ctl.dq_drained, 8);
    mbar_init(&ctl.drain, 1);
    mbar_init(&ctl.fin, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ctl.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = ctl.tmem_slot;

  // Rows of query tile i that hold a row of the sequence.
  const int G = p.G, tpt = p.tpt;
  auto q_rows = [=](int n, int i) { return min(tpt, n - i * tpt) * G; };

  if (warp == 10) {
    // ------------------------------------------------------------------ scheduler
    griddep_wait();
    int ii = 0;
    bool ok = true;
    SeqBwdItem it{};
    auto publish = [&]() -> bool {
      const int s = ii % NI;
      bool free = true;
      if (ii >= NI) free = mbar_wait(&ctl.item_empty[s], ((ii / NI) - 1) & 1, wc, kRSiteItemEmpty);
      if (!__all_sync(0xffffffffu, free)) return false;
      if (lane == 0) {
        ctl.items[s] = it;
        mbar_arrive(&ctl.item_full[s]);
      }
      ++ii;
      return true;
    };
    BlockOrder<kHeldBwd> order;
    order.load(ctl.held, p.cu, p.B, p.T, 128, lane);
    int w = blockIdx.x;
    BlockAt at;
    for (int k = 0; ok && w >= 0; ++k) {
      const int ws = SPLIT ? w / p.split : w;
      [[maybe_unused]] const int s = SPLIT ? w - ws * p.split : 0;
      if (order.find(p.cu, p.B, p.T, p.Hkv, p.head_group, 128, ws, lane, at)) {
        it.row0 = min(max(p.cu[at.b], 0), p.T);
        it.n = rows_of(p.cu, p.T, at.b);
        it.kvh = at.kvh;
        // Causal: key tile 0 has the most query tiles.
        it.j = (it.n + 127) / 128 - 1 - at.level;
        query_range(p, it.n, it.j, it.i0, it.n_it);
        if constexpr (SPLIT) {  // part s of at most `split`
          const int parts = min(p.split, it.n_it), a = it.n_it * s / parts, e = it.n_it * (s + 1) / parts;
          it.part = s;
          it.i0 += a;
          it.n_it = s < parts ? e - a : 0;
        }
        it.qt0 = tile_base(p, at.b);
        it.valid = 1;
        if (it.n_it > 0) ok = publish();
      }
      // The next index only once the item before this one is done with.
      if (ok && ii >= 2)
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.item_empty[(ii - 2) % NI], ((ii - 2) / NI) & 1, wc, kRSiteItemEmpty));
      if (!ok) break;
      if (lane == 0) {
        fence_proxy_async_smem();  // the response was read before it is written again
        mbar_arrive_expect_tx(&ctl.clc_full, 16);
        clc_try_cancel(&ctl.clc_response, &ctl.clc_full);
      }
      __syncwarp();
      volatile int no_abort = 0;  // the response always lands before the CTA leaves
      WaitCtl cw{p.status, &no_abort, p.wait_ns};
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.clc_full, k & 1, cw, kRSiteClc));
      if (!ok) break;
      w = lane == 0 ? clc_index(&ctl.clc_response) : 0;
      w = __shfl_sync(0xffffffffu, w, 0);
    }
    it.valid = 0;
    if (ok) publish();
  } else if (warp == 11) {
    // ------------------------------------------------------------------ rows of no sequence
    unsigned int par = 0;  // bits 0-1 kv_raw, 2-3 qdo_raw, 4-5 q_raw
    bool ok = true;
    int gs = 0;
    auto zero = [&](uint8_t* tile, int from) {
      for (int r = from + (lane >> 3); r < 128; r += 4)
        for (int c = 0; c < C::KCH; ++c)
          *reinterpret_cast<uint4*>(tile + c * C::CHUNK + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
    };
    auto raw = [&](uint64_t* bar, int bit) -> bool {
      const bool r = __all_sync(0xffffffffu, mbar_wait(bar, par >> bit & 1, wc, kRSiteFix)) != 0;
      par ^= 1u << bit;
      return r;
    };
    auto done = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.item_full[k % NI], (k / NI) & 1, wc, kRSiteItem));
      if (!ok) break;
      const SeqBwdItem it = ctl.items[k % NI];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.item_empty[k % NI]);
      if (!it.valid) break;
      const int b = k % C::KVB, keys = it.n - it.j * 128;
      if (keys < 128) {
        ok = raw(&ctl.kv_raw[b], b);
        if (!ok) break;
        zero(sK + b * C::TILE, keys);
        zero(sV + b * C::TILE, keys);
        done(&ctl.kv_full[b]);
      }
      for (int x = 0; x < it.n_it && ok; ++x, ++gs) {
        const int rows = q_rows(it.n, it.i0 + x), st = gs % C::ST;
        if (rows >= 128) continue;
        if constexpr (C::PIPE) {
          ok = raw(&ctl.qdo_raw[st], 2 + st);
          if (!ok) break;
          zero(sQ + st * C::TILE, rows);
          zero(sdO + st * C::TILE, rows);
          done(&ctl.qdo_full[st]);
        } else {
          ok = raw(&ctl.q_raw[st], 4 + st);
          if (!ok) break;
          zero(sQ + st * C::TILE, rows);
          done(&ctl.q_full[st]);
          ok = raw(&ctl.qdo_raw[st], 2 + st);
          if (!ok) break;
          zero(sdO + st * C::TILE, rows);
          done(&ctl.qdo_full[st]);
        }
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmdO);
      const uint64_t keep = policy_evict_last();
      const uint32_t q_bytes = C::KCH * 128 * G * tpt;
      // Loads issued per slot: count, and whether (and how often) it was the raw barrier.
      unsigned int par = 0, is_raw = 0;  // bits as in the fix warp
      int gs = 0, gq = 0, kvs = 0;
      bool ok = true;
      auto bar_for = [&](bool fix, uint64_t* raw, uint64_t* full, int bit) -> uint64_t* {
        is_raw = fix ? is_raw | (1u << bit) : is_raw & ~(1u << bit);
        if (fix) par ^= 1u << bit;
        return fix ? raw : full;
      };
      griddep_wait();
      // K and V of item k.  (The test hook skips them: a consumer's wait then runs out.)
      auto load_kv = [&](const SeqBwdItem& it, int k) -> bool {
        if (p.fault == 1) return true;
        const int b = k % C::KVB, u = k / C::KVB;
        if (u > 0 && !mbar_wait(&ctl.kv_empty[b], (u - 1) & 1, wc, kRSiteProd)) return false;
        uint64_t* bar = bar_for(it.n - it.j * 128 < 128, &ctl.kv_raw[b], &ctl.kv_full[b], b);
        mbar_arrive_expect_tx(bar, 2 * C::TILE);
        for (int c = 0; c < C::KCH; ++c) {
          tma_load_3d(sK + b * C::TILE + c * C::CHUNK, &tmK, bar, c * 64, it.row0 + it.j * 128, it.kvh);
          tma_load_3d(sV + b * C::TILE + c * C::CHUNK, &tmV, bar, c * 64, it.row0 + it.j * 128, it.kvh);
        }
        kvs = k + 1;
        return true;
      };
      for (int k = 0; ok; ++k) {
        if (!mbar_wait(&ctl.item_full[k % NI], (k / NI) & 1, wc, kRSiteItem)) { ok = false; break; }
        const SeqBwdItem it = ctl.items[k % NI];
        mbar_arrive(&ctl.item_empty[k % NI]);
        if (!it.valid) break;
        // Two buffers: K, V ahead of the first (Q, dO); one: behind it, as the buffer is
        // released by the last product of the item before.
        if (C::KVB == 2 || k == 0) ok = load_kv(it, k);
        for (int x = 0; x < it.n_it && ok; ++x) {
          const int st = gs % C::ST, i = it.i0 + x;
          const int tok = it.row0 + i * tpt;
          const bool fix = q_rows(it.n, i) < 128;
          const size_t stat = (static_cast<size_t>(it.kvh) * p.tiles + it.qt0 + i) * 128;
          if constexpr (!C::PIPE) {
            if (gs >= C::ST && !mbar_wait(&ctl.q_empty[st], ((gs / C::ST) - 1) & 1, wc, kRSiteProd)) { ok = false; break; }
            uint64_t* bar = bar_for(fix, &ctl.q_raw[st], &ctl.q_full[st], 4 + st);
            mbar_arrive_expect_tx(bar, q_bytes + 1024);
            bulk_load(sLD + st * 256, p.Lg + stat, 512, bar);
            bulk_load(sLD + st * 256 + 128, p.Dg + stat, 512, bar);
            for (int c = 0; c < C::KCH; ++c)
              tma_load_3d_hint(sQ + st * C::TILE + c * C::CHUNK, &tmQ, bar, c * 64, it.kvh * G, tok, keep);
            ++gq;
          }
          if (gs >= C::ST && !mbar_wait(&ctl.qdo_empty[st], ((gs / C::ST) - 1) & 1, wc, kRSiteProd)) { ok = false; break; }
          uint64_t* bar = bar_for(fix, &ctl.qdo_raw[st], &ctl.qdo_full[st], 2 + st);
          mbar_arrive_expect_tx(bar, C::PIPE ? 2 * q_bytes + 1024 : q_bytes);
          if constexpr (C::PIPE) {
            bulk_load(sLD + st * 256, p.Lg + stat, 512, bar);
            bulk_load(sLD + st * 256 + 128, p.Dg + stat, 512, bar);
          }
          for (int c = 0; c < C::KCH; ++c) {
            if constexpr (C::PIPE)
              tma_load_3d_hint(sQ + st * C::TILE + c * C::CHUNK, &tmQ, bar, c * 64, it.kvh * G, tok, keep);
            tma_load_3d_hint(sdO + st * C::TILE + c * C::CHUNK, &tmdO, bar, c * 64, it.kvh * G, tok, keep);
          }
          ++gs;
          if (C::KVB == 1 && k > 0 && x == 0) ok = load_kv(it, k);
        }
      }
      // Every copy that was issued lands before the CTA leaves, on a timeout too.
      volatile int no_abort = 0;
      WaitCtl dw{p.status, &no_abort, 100000000ull};
      auto landed = [&](int slot, int count, uint64_t* raw, uint64_t* full, int bit) {
        if (is_raw >> bit & 1) mbar_wait(raw + slot, (par >> bit & 1) ^ 1, dw, kRSiteDrain);
        else mbar_wait(full + slot, count & 1, dw, kRSiteDrain);
      };
      for (int q = max(0, gs - C::ST); q < gs; ++q)
        landed(q % C::ST, q / C::ST, ctl.qdo_raw, ctl.qdo_full, 2 + q % C::ST);
      if (!C::PIPE)
        for (int q = max(0, gq - C::ST); q < gq; ++q) landed(q % C::ST, q / C::ST, ctl.q_raw, ctl.q_full, 4 + q % C::ST);
      for (int k = max(0, kvs - C::KVB); k < kvs; ++k)
        landed(k % C::KVB, k / C::KVB, ctl.kv_raw, ctl.kv_full, k % C::KVB);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_kk = idesc_f16(128, 128, BF16, false, false);  // S^T, dP^T
      constexpr uint32_t id_tb = idesc_f16(128, D, BF16, false, true);     // dV, dK (B MN-major)
      constexpr uint32_t id_dq = idesc_f16(128, D, BF16, true, true);      // dQ (A, B MN-major)
      const uint32_t aK = smem_u32(sK), aV = smem_u32(sV), aQ = smem_u32(sQ), adO = smem_u32(sdO), aDS = smem_u32(sDS);
      const uint64_t kK = sdesc_sw128(aK, 16, 1024), kV = sdesc_sw128(aV, 16, 1024);
      const uint64_t kQ = sdesc_sw128(aQ, 16, 1024), kdO = sdesc_sw128(adO, 16, 1024);
      const uint64_t mQ = sdesc_sw128(aQ, C::CHUNK, 1024), mdO = sdesc_sw128(adO, C::CHUNK, 1024);
      const uint64_t mK = sdesc_sw128(aK, C::CHUNK, 1024), mDS = sdesc_sw128(aDS, C::CHUNK, 1024);
      auto mma_s = [&](int st, uint32_t kvo) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
          umma_ss(tbase + C::C_S, sdesc_add(kK, kvo + off), sdesc_add(kQ, st * C::TILE + off), id_kk, kk > 0);
        }
        umma_commit(&ctl.s_full);
      };
      auto mma_dp = [&](int st, uint32_t kvo) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
          umma_ss(tbase + C::C_DP, sdesc_add(kV, kvo + off), sdesc_add(kdO, st * C::TILE + off), id_kk, kk > 0);
        }
        umma_commit(&ctl.dp_full);
      };
      auto mma_dv = [&](int st, bool first) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ts(tbase + C::C_DV, tbase + C::C_P(kk >> 2) + (kk & 3) * 8, sdesc_add(mdO, st * C::TILE + kk * 2048),
                  id_tb, (!first || kk > 0) ? 1u : 0u);
      };
      auto mma_dq = [&](uint32_t kvo) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ss(tbase + C::C_DQ, sdesc_add(mDS, kk * 2048), sdesc_add(mK, kvo + kk * 2048), id_dq, kk > 0);
        umma_commit(&ctl.dq_full);
      };
      auto mma_dk = [&](int st, bool first) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ts(tbase + C::C_DK, tbase + C::C_DS(kk >> 2) + (kk & 3) * 8, sdesc_add(mQ, st * C::TILE + kk * 2048),
                  id_tb, (!first || kk > 0) ? 1u : 0u);
        umma_commit(C::PIPE ? &ctl.qdo_empty[st] : &ctl.q_empty[st]);
      };
      auto wait = [&](uint64_t* bar, int phase, uint32_t site) -> bool {
        const bool r = mbar_wait(bar, phase & 1, wc, site);
        tc_fence_after();
        return r;
      };
      bool ok = true;
      int gs = 0;  // query steps so far
      for (int k = 0; ok; ++k) {
        if (!mbar_wait(&ctl.item_full[k % NI], (k / NI) & 1, wc, kRSiteItem)) { ok = false; break; }
        const int n_it = ctl.items[k % NI].n_it;
        const bool valid = ctl.items[k % NI].valid != 0;
        mbar_arrive(&ctl.item_empty[k % NI]);
        if (!valid) break;
        const int b = k % C::KVB;
        const uint32_t kvo = static_cast<uint32_t>(b * C::TILE);
        if (!wait(&ctl.kv_full[b], k / C::KVB, kRSiteMmaKV)) { ok = false; break; }
        if constexpr (!C::PIPE) {
          // D = 128: no free columns; each step in order -- S^T, dP^T (once the dQ partial in
          // its columns is drained), dV, dQ, dK.
          for (int it = 0; it < n_it && ok; ++it, ++gs) {
            const int st = gs % C::ST;
            if (!(ok = wait(&ctl.q_full[st], gs / C::ST, kRSiteMmaQ))) break;
            mma_s(st, kvo);
            if (gs > 0 && !(ok = wait(&ctl.dq_drained, gs - 1, kRSiteMmaDrained))) break;
            if (!(ok = wait(&ctl.qdo_full[st], gs / C::ST, kRSiteMmaQ))) break;
            mma_dp(st, kvo);
            if (!(ok = wait(&ctl.p_ready, gs, kRSiteMmaP))) break;
            // An item's first dV and dK overwrite the accumulators: read out by then.
            if (k > 0 && it == 0 && !(ok = wait(&ctl.acc_free, k - 1, kRSiteMmaAcc))) break;
            mma_dv(st, it == 0);
            if (!(ok = wait(&ctl.ds_ready, gs, kRSiteMmaDS))) break;
            mma_dq(kvo);
            if (it == n_it - 1) umma_commit(&ctl.kv_empty[b]);
            mma_dk(st, it == 0);
          }
        } else {
          // D = 64: the next step's S^T right behind this one's dV, its dP^T behind this one's dK.
          if (!(ok = wait(&ctl.qdo_full[gs % C::ST], gs / C::ST, kRSiteMmaQ))) break;
          mma_s(gs % C::ST, kvo);
          mma_dp(gs % C::ST, kvo);
          for (int it = 0; it < n_it && ok; ++it, ++gs) {
            const int st = gs % C::ST;
            if (!(ok = wait(&ctl.p_ready, gs, kRSiteMmaP))) break;
            if (k > 0 && it == 0 && !(ok = wait(&ctl.acc_free, k - 1, kRSiteMmaAcc))) break;
            mma_dv(st, it == 0);
            if (it + 1 < n_it) {
              if (!(ok = wait(&ctl.qdo_full[(gs + 1) % C::ST], (gs + 1) / C::ST, kRSiteMmaQ))) break;
              mma_s((gs + 1) % C::ST, kvo);
            }
            if (!(ok = wait(&ctl.ds_ready, gs, kRSiteMmaDS))) break;
            if (gs > 0 && !(ok = wait(&ctl.dq_drained, gs - 1, kRSiteMmaDrained))) break;
            mma_dq(kvo);
            if (it == n_it - 1) umma_commit(&ctl.kv_empty[b]);
            mma_dk(st, it == 0);
            if (it + 1 < n_it) mma_dp((gs + 1) % C::ST, kvo);
          }
        }
        if (ok) umma_commit(&ctl.drain);  // the item's dK and dV are final once this lands
      }
      umma_commit(&ctl.fin);
      volatile int no_abort = 0;
      WaitCtl dw{p.status, &no_abort, p.wait_ns};
      mbar_wait(&ctl.fin, 0, dw, kRSiteMmaDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ compute
    griddep_wait();  // the accumulator was zeroed by the preprocess
    const int g = warp >> 2;  // warpgroup: query columns 64 g .. 64 g + 63
    const int wq = warp & 3;  // tensor-memory lane quadrant
    const int r = wq * 32 + lane;  // key row (P^T, dS^T) / query row (dQ)
    const uint32_t lb = static_cast<uint32_t>(wq * 32);
    const float sl2 = p.scale_log2;
    const int qoff = 64 * g;
    const uint32_t wg_bar = 1 + g;
    bool ok = true;
    int gs = 0;
    float pr[64];  // this warpgroup's P^T of a step
    // Every wait ends in a warpgroup-wide vote: on a timeout all 128 threads leave together,
    // and no named barrier is left waiting.
    auto stage_p = [&](int gp, int ip, int key, int n) -> bool {
      const int st = gp % C::ST;
      const float4* L4 = reinterpret_cast<const float4*>(sLD + st * 256 + qoff);
      uint64_t* ld = C::PIPE ? &ctl.qdo_full[st] : &ctl.q_full[st];
      if (!named_bar_and(wg_bar, 128, mbar_wait(ld, (gp / C::ST) & 1, wc, kRSiteCmpQ))) return false;
      if (!named_bar_and(wg_bar, 128, mbar_wait(&ctl.s_full, gp & 1, wc, kRSiteCmpS))) return false;
      tc_fence_after();
      // Query columns [q_lo, q_hi) of the tile see this key (row = token * G + head).
      const int ahead = key - ip * tpt;  // the key's position counted from the tile's first token
      int q_lo = 0, q_hi = 128;
      if (p.causal) q_lo = min(max(ahead, 0), 128) * G;
      if (p.window > 0) q_hi = ahead + p.window >= 128 ? 128 : max(ahead + p.window, 0) * G;
      if (key >= n) q_hi = 0;
      const bool masked = __any_sync(0xffffffffu, q_lo > qoff || q_hi < qoff + 64);
      const uint64_t sl2x2 = f2_pack(sl2, sl2);
      uint32_t srr[2][32];
      tmem_ld32(tmem_addr(tbase, lb, C::C_S + qoff), srr[0]);
      tmem_ld32(tmem_addr(tbase, lb, C::C_S + qoff + 32), srr[1]);
      tmem_wait_ld();
      reg_fence(srr[0]);
      reg_fence(srr[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float4 l4 = L4[c * 8 + v];
          const uint32_t* sr = &srr[c][v * 4];
          const int q0 = c * 32 + v * 4;
          float x0, x1, x2, x3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[0]), __uint_as_float(sr[1])), sl2x2, f2_pack(-l4.x, -l4.y)), x0, x1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2]), __uint_as_float(sr[3])), sl2x2, f2_pack(-l4.z, -l4.w)), x2, x3);
          pr[q0 + 0] = ex2_approx(x0);
          pr[q0 + 1] = ex2_approx(x1);
          pr[q0 + 2] = ex2_approx(x2);
          pr[q0 + 3] = ex2_approx(x3);
        }
      }
      if (masked) {
#pragma unroll
        for (int q = 0; q < 64; ++q)
          if (qoff + q < q_lo || qoff + q >= q_hi) pr[q] = 0.f;
      }
      uint32_t pk[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) pk[e] = pack2<BF16>(pr[2 * e], pr[2 * e + 1]);
      tmem_st32(tmem_addr(tbase, lb, C::C_P(g)), pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.p_ready);
      return true;
    };
    auto stage_ds = [&](int gd) -> bool {
      const float4* D4 = reinterpret_cast<const float4*>(sLD + (gd % C::ST) * 256 + 128 + qoff);
      if (!named_bar_and(wg_bar, 128, mbar_wait(&ctl.dp_full, gd & 1, wc, kRSiteCmpDP))) return false;
      tc_fence_after();
      if (gd > 0) {
        // This warpgroup's dS^T chunk (and at D = 128 its half of the step before's dO tile)
        // staged that step's dQ reduce: the copies have finished reading it.
        if (r == 0) {
          tma_store_wait_read();
          if constexpr (!C::PIPE) mbar_arrive(&ctl.qdo_empty[(gd - 1) % C::ST]);
        }
        named_bar_sync(wg_bar, 128);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dr[32];
        tmem_ld32(tmem_addr(tbase, lb, C::C_DP + qoff + 32 * c), dr);
        tmem_wait_ld();
        reg_fence(dr);
        uint32_t dsk[16];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float4 d4 = D4[c * 8 + v];
          const int q0 = c * 32 + v * 4;
          const uint64_t t01 = f2_sub(f2_pack(__uint_as_float(dr[v * 4]), __uint_as_float(dr[v * 4 + 1])), f2_pack(d4.x, d4.y));
          const uint64_t t23 = f2_sub(f2_pack(__uint_as_float(dr[v * 4 + 2]), __uint_as_float(dr[v * 4 + 3])), f2_pack(d4.z, d4.w));
          float a0, a1, a2, a3;
          f2_unpack(f2_mul(f2_pack(pr[q0], pr[q0 + 1]), t01), a0, a1);
          f2_unpack(f2_mul(f2_pack(pr[q0 + 2], pr[q0 + 3]), t23), a2, a3);
          dsk[2 * v] = pack2<BF16>(a0, a1);
          dsk[2 * v + 1] = pack2<BF16>(a2, a3);
        }
        tmem_st16(tmem_addr(tbase, lb, C::C_DS(g) + 16 * c), dsk);
#pragma unroll
        for (int uu = 0; uu < 4; ++uu) {
          const int u = c * 4 + uu;
          *reinterpret_cast<uint4*>(sDS + g * C::CHUNK + r * 128 + ((u ^ (r & 7)) << 4)) =
              make_uint4(dsk[4 * uu], dsk[4 * uu + 1], dsk[4 * uu + 2], dsk[4 * uu + 3]);
        }
      }
      fence_proxy_async_smem();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.ds_ready);
      return true;
    };
    auto stage_dq = [&](int gq, int tile, int kvh) -> bool {
      if (!named_bar_and(wg_bar, 128, mbar_wait(&ctl.dq_full, gq & 1, wc, kRSiteCmpDQ))) return false;
      tc_fence_after();
      // dQ partial: tensor memory -> 128 x 32-float tiles in shared memory -> one TMA
      // reduce-add each into the tile's rows of the accumulator.
      constexpr int HALF = D / 2, NCH = HALF / 32;
      uint8_t* stage = sDS + g * C::CHUNK;
      if constexpr (C::PIPE) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t q16[16];
          tmem_ld16(tmem_addr(tbase, lb, C::C_DQ + g * HALF + 16 * h), q16);
          tmem_wait_ld();
          reg_fence(q16);
          if (h == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.dq_drained);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(stage + r * 128 + (((4 * h + u) ^ (r & 7)) << 4)) =
                make_uint4(q16[4 * u], q16[4 * u + 1], q16[4 * u + 2], q16[4 * u + 3]);
        }
        fence_proxy_async_smem();
        named_bar_sync(wg_bar, 128);
        if (r == 0) {
          tma_reduce_add_3d(&tmdQ, stage, g * HALF, tile * 128, kvh);
          tma_store_commit();
        }
        __syncwarp();
      } else {
        uint32_t qr[NCH][32];
#pragma unroll
        for (int c = 0; c < NCH; ++c) tmem_ld32(tmem_addr(tbase, lb, C::C_DQ + g * HALF + 32 * c), qr[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < NCH; ++c) reg_fence(qr[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.dq_drained);
        // The second tile goes to this warpgroup's half of the step's dO tile (its readers
        // have completed), so that both reduces leave together.
        uint8_t* stg[2] = {stage, sdO + (gq % C::ST) * C::TILE + g * C::CHUNK};
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(stg[c] + r * 128 + ((u ^ (r & 7)) << 4)) =
                make_uint4(qr[c][4 * u], qr[c][4 * u + 1], qr[c][4 * u + 2], qr[c][4 * u + 3]);
        fence_proxy_async_smem();
        named_bar_sync(wg_bar, 128);
        if (r == 0) {
          tma_reduce_add_3d(&tmdQ, stg[0], g * HALF, tile * 128, kvh);
          tma_reduce_add_3d(&tmdQ, stg[1], g * HALF + 32, tile * 128, kvh);
          tma_store_commit();
        }
        __syncwarp();
      }
      return true;
    };
    for (int k = 0; ok; ++k) {
      if (!named_bar_and(wg_bar, 128, mbar_wait(&ctl.item_full[k % NI], (k / NI) & 1, wc, kRSiteItem))) break;
      const SeqBwdItem it = ctl.items[k % NI];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.item_empty[k % NI]);
      if (!it.valid) break;
      const int key = it.j * 128 + r;
      const int g0 = gs;
      if constexpr (!C::PIPE) {
        for (int x = 0; x < it.n_it && ok; ++x)
          ok = stage_p(g0 + x, it.i0 + x, key, it.n) && stage_ds(g0 + x) && stage_dq(g0 + x, it.qt0 + it.i0 + x, it.kvh);
      } else {
        ok = stage_p(g0, it.i0, key, it.n);
        for (int x = 0; x < it.n_it && ok; ++x) {
          ok = stage_ds(g0 + x);
          if (ok && x + 1 < it.n_it) ok = stage_p(g0 + x + 1, it.i0 + x + 1, key, it.n);
          if (ok) ok = stage_dq(g0 + x, it.qt0 + it.i0 + x, it.kvh);
        }
      }
      gs = g0 + it.n_it;
      if (!ok) break;
      // dV (warpgroup 0) and dK (warpgroup 1): out of tensor memory, the columns handed to the
      // next item's products, then stored.
      ok = named_bar_and(wg_bar, 128, mbar_wait(&ctl.drain, k & 1, wc, kRSiteCmpDQ));
      if (!ok) break;
      tc_fence_after();
      const float mul = g ? p.scale : 1.0f;
      uint16_t* row = g ? p.dK + (it.row0 + key) * p.dk_row + it.kvh * p.dk_head
                        : p.dV + (it.row0 + key) * p.dv_row + it.kvh * p.dv_head;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t rr[32];
        tmem_ld32(tmem_addr(tbase, lb, (g ? C::C_DK : C::C_DV) + 32 * c), rr);
        tmem_wait_ld();
        reg_fence(rr);
        if (c == D / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.acc_free);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int f = 0; f < 4; ++f)
            w[f] = pack2<BF16>(__uint_as_float(rr[8 * e + 2 * f]) * mul, __uint_as_float(rr[8 * e + 2 * f + 1]) * mul);
          if (!SPLIT && key < it.n && c * 32 + 8 * e < p.d)
            *reinterpret_cast<uint4*>(row + c * 32 + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (SPLIT && key < it.n) {
          float4* dst = reinterpret_cast<float4*>(
              p.kv_part + (((static_cast<size_t>(it.part) * 2 + g) * p.T + it.row0 + key) * p.Hkv + it.kvh) * D + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(rr[4 * e]), __uint_as_float(rr[4 * e + 1]),
                                 __uint_as_float(rr[4 * e + 2]), __uint_as_float(rr[4 * e + 3]));
        }
      }
    }
    if (r == 0) tma_store_wait_all();  // the reductions complete before shared memory goes away
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace fa2
