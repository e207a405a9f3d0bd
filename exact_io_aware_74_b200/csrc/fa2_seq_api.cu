// Host side of the packed-sequence and paged-cache entry points of libfa2.so:
// argument validation and launches.  Declarations and contracts are in include/fa2.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/fa2.h"
#include "fa2_host.h"
#include "fa2_paged.cuh"
#include "fa2_seq_bwd.cuh"
#include "fa2_seq_host.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kMaxFwdHeadDim = 256;
constexpr int kMaxBwdHeadDim = 128;
constexpr int kMaxGroup = 128;  // query heads to a key/value head: rows of one query tile

int check_sizes(int B, int T, int H, int Hkv, int d, int max_d) {
  if (B < 1 || T < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > kMaxGroup) return FA2_ERR_INVALID_ARG;
  if (B > (1 << 24) || T > (1 << 30) || H > 32767) return FA2_ERR_INVALID_ARG;
  if (d < 8 || d > max_d || d % 8 != 0) return FA2_ERR_UNSUPPORTED;
  return FA2_OK;
}

int check_mode(float scale, int causal, int window, int dtype) {
  if (causal != 0 && causal != 1) return FA2_ERR_INVALID_ARG;
  if (window < 0 || (window > 0 && causal != 1)) return FA2_ERR_INVALID_ARG;
  if (dtype != FA2_FP16 && dtype != FA2_BF16) return FA2_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA2_ERR_INVALID_ARG;
  return FA2_OK;
}

bool stride_ok(long long s, long long least) { return s >= least && s % 8 == 0 && s < (1ll << 38); }

// A packed tensor of `heads` heads of d columns.  A stride whose axis has one entry is
// not read and may be anything.
bool packed_ok(const fa2_packed* x, int T, int heads, int d) {
  return x && x->data && aligned(x->data, 16) && (T <= 1 || stride_ok(x->stride_row, d)) &&
         (heads <= 1 || stride_ok(x->stride_head, d));
}
bool cache_ok(const fa2_cache* x, int blocks, int heads, int rows, int d) {
  return x && x->data && aligned(x->data, 16) && (blocks <= 1 || stride_ok(x->stride_block, d)) &&
         (heads <= 1 || stride_ok(x->stride_head, d)) && (rows <= 1 || stride_ok(x->stride_row, d));
}

// Sequences that may hold a partial block: the empty ones too where the order of the blocks
// keeps a place for each (BlockOrder).
int partial_blocks(int B, int T, int held) { return B > held ? B : std::min(B, T); }

// Key/value heads to a group of the item order: as many equal groups as leave each `waves`
// waves of items.  Fewer heads leave SMs without work where a group's longest items start last,
// more let the heads' rows fall out of L2.  Measured on B200 (heads to a group, replayed graphs;
// the calls of 1 ms and more vary by 5 % with the power limit): backward of 14k tokens, d = 128, 920
// items of very different length: 1: 1748, 2: 1738, 3: 1761, 4: 1649, 8 (the rule): 1560 to 1630 us; of
// 4k tokens, d = 64, 4 heads: 1: 111, 2: 100, 4 (the rule): 82 us; of 8 x 4096 tokens, d = 128, 16
// heads, 4200 items: 1: 1989, 3 (the rule): 2011 to 2059, 5: 2140, 8: 2183, 16: 2466 us.  Forward of 15k
// tokens, d = 64, 1050 items: 1: 158, 2: 143, 3: 147, 4: 134, 8 (the rule): 128 us; of 22k tokens,
// d = 128, 2800 items: 1: 1209, 2: 1164, 3 (the rule): 1185, 4: 1211, 8: 1213 us.
int head_group(long long items, int waves, int Hkv, int n_sm) {
  const long long groups = std::min<long long>(Hkv, std::max(1ll, items / (static_cast<long long>(waves) * n_sm)));
  return static_cast<int>((Hkv + groups - 1) / groups);
}

// ---- forward over packed sequences and paged caches ----

// [T][heads][d] as a 3-D map (column, head, row) or (column, row, head).  The stride of
// an axis with one entry is not the caller's.
bool map_packed(CUtensorMap* m, const fa2_packed* x, int T, int heads, int d, int dtype, bool rows_inside,
                uint32_t box_rows, uint32_t box_heads) {
  const uint64_t row = T > 1 ? x->stride_row * 2 : d * 2, head = heads > 1 ? x->stride_head * 2 : d * 2;
  const fa2::MapType ty = dtype == FA2_BF16 ? fa2::MapType::kBF16 : fa2::MapType::kF16;
  const uint64_t D = d, N = T, H = heads;
  if (rows_inside) {
    const uint64_t dims[3] = {D, N, H}, strides[2] = {row, head};
    const uint32_t box[3] = {64, box_rows, box_heads};
    return fa2::host_encode_map(m, ty, x->data, 3, dims, strides, box);
  }
  const uint64_t dims[3] = {D, H, N}, strides[2] = {head, row};
  const uint32_t box[3] = {64, box_heads, box_rows};
  return fa2::host_encode_map(m, ty, x->data, 3, dims, strides, box);
}

bool map_cache(CUtensorMap* m, const fa2_cache* x, int blocks, int heads, int rows, int d, int dtype) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(rows), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(blocks)};
  const uint64_t any = static_cast<uint64_t>(d) * 2;
  const uint64_t strides[3] = {rows > 1 ? static_cast<uint64_t>(x->stride_row) * 2 : any,
                               heads > 1 ? static_cast<uint64_t>(x->stride_head) * 2 : any,
                               blocks > 1 ? static_cast<uint64_t>(x->stride_block) * 2 : any};
  const uint32_t box[4] = {64, static_cast<uint32_t>(std::min(rows, 128)), 1, 1};
  return fa2::host_encode_map(m, dtype == FA2_BF16 ? fa2::MapType::kBF16 : fa2::MapType::kF16, x->data, 4, dims,
                              strides, box);
}

fa2::SeqParams seq_params(const fa2_packed* O, float* LSE, const int* cu, unsigned int* st, int B, int T, int H,
                          int Hkv, int d, float scale, int causal, int window) {
  fa2::SeqParams p{};
  p.O = static_cast<uint16_t*>(O->data);
  p.o_row = O->stride_row;
  p.o_head = O->stride_head;
  p.LSE = LSE;
  p.cu = cu;
  p.status = st;
  p.wait_ns = fa2::host_wait_ns();
  p.fault = fa2::host_fault();
  p.B = B, p.T = T, p.Hkv = Hkv, p.G = H / Hkv, p.d = d, p.tpt = 128 / p.G;
  p.causal = causal, p.window = std::min(window, 1 << 30);  // longer than any sequence
  p.scale_log2 = scale * 1.4426950408889634f;
  return p;
}

// Form of a paged call's items, by the rows that the requests bring on average: two query
// tiles of 128 rows (prompts, chunks), one, or 16 rows with the products' operands swapped
// (decode steps; d <= 128).  Every form is right for every batch.  Measured on B200 (replayed graphs,
// single tokens, 8 key/value heads, blocks of 16), 16 rows against one tile:
//   64 requests of up to 6000 tokens, 1, 4, 16 heads to a group: d = 64: 121, 123, 139 us against 147,
//     148, 149; d = 128: 166, 170, 174 against 163, 165, 171
//   4 heads to a group: 64 requests of up to 8192 tokens: d = 64: 170 to 183 against 193 to 197, d = 128:
//     225 against 218; of up to 700: d = 64: 41.2 against 39.5, d = 128: 47.3 against 44.1; 4 of up to
//     32768: d = 64: 56 against 62, d = 128: 73.5 against 71.5; 4 of up to 700: 14.0 against 13.3, 14.4
//     against 13.6
// So 16 rows gain 7 to 18 % on long caches of 64-column heads and cost 1 to 7 % elsewhere, where the
// rule, which looks at the rows alone, takes them all the same.  (The swapped form with 32 rows spilled
// and took 660 us where one tile took 203: it was dropped.)
int paged_form(int B, int T, int G, int d) {
  if (d > 128) return 1;
  const long long rows = static_cast<long long>(T) * G, b = B;
  if (G <= 16 && rows <= 16 * b) return 16;
  return T > 128 / G * b ? 2 : 1;
}
int form_tiles(int form) { return form == 2 ? 2 : 1; }           // 128-row tiles of a partial slot
int form_tokens(int form, int G) { return (form == 16 ? 16 : 128) / G; }  // tokens to a tile

// Float partials of the shares, two slots each: O, then LSE, then what is to be merged.
size_t paged_opart_bytes(int grid, int qt, int d) {
  return static_cast<size_t>(grid) * 2 * qt * 128 * fa2::seq_tile_dim(d) * 4;
}
size_t paged_bytes(int grid, int qt, int d) {
  return paged_opart_bytes(grid, qt, d) + static_cast<size_t>(grid) * (2 * qt * 128 * 4 + sizeof(int4));
}

// ---- backward ----

constexpr long long kBwdWaves = 3;

int bwd_tile_dim(int d) { return d <= 64 ? 64 : 128; }

// Query tiles of one key/value head: each sequence's last one may be partial.
long long bwd_tiles(int B, int T, int G) { return T / (128 / G) + static_cast<long long>(B); }

// Work items of the backward, and the parts that a key tile's query tiles are cut into: as
// many as give about three waves of items on a B200's 148 SMs, eight at most.
long long bwd_items(int B, int T, int Hkv) {
  return (T / 128 + static_cast<long long>(partial_blocks(B, T, fa2::kHeldBwd))) * Hkv;
}
int bwd_split(int B, int T, int Hkv) {
  return static_cast<int>(std::min(8ll, std::max(1ll, kBwdWaves * 148 / std::max(1ll, bwd_items(B, T, Hkv)))));
}

// Workspace: D and LSE * log2 e per row, then the float dQ accumulator.
size_t bwd_stat_bytes(int B, int T, int H, int Hkv) {
  return static_cast<size_t>(bwd_tiles(B, T, H / Hkv)) * Hkv * 128 * 4;  // a multiple of 512
}

}  // namespace

extern "C" {

int fa2_fwd_varlen(const fa2_packed* Q, const fa2_packed* K, const fa2_packed* V,
                   const fa2_packed* O, float* LSE, const int* cu_seqlens, int B, int T, int H,
                   int Hkv, int d, float scale, int causal, int window, int dtype,
                   fa2_stream_t stream) {
  int rc = check_sizes(B, T, H, Hkv, d, kMaxFwdHeadDim);
  if (rc == FA2_OK) rc = check_mode(scale, causal, window, dtype);
  if (rc != FA2_OK) return rc;
  if (T == 0) return FA2_OK;
  if (!packed_ok(Q, T, H, d) || !packed_ok(K, T, Hkv, d) || !packed_ok(V, T, Hkv, d) ||
      !packed_ok(O, T, H, d) || !LSE || !aligned(LSE, 4) || !cu_seqlens || !aligned(cu_seqlens, 4))
    return FA2_ERR_INVALID_ARG;
  for (const fa2_packed* x : {Q, K, V})
    if (x->data == O->data || x->data == LSE) return FA2_ERR_INVALID_ARG;
  int dev, n_sm;
  unsigned int* st;
  rc = fa2::host_device(&dev, &n_sm, &st);
  if (rc != FA2_OK) return rc;
  const int G = H / Hkv, tpt = 128 / G;
  // Items there could be: every sequence's last block may be partial.
  const auto items = [&](int qt) {
    return (static_cast<long long>(T) / (qt * tpt) + partial_blocks(B, T, fa2::kHeld)) * Hkv;
  };
  // Two query tiles to a CTA; one (twice the CTAs) where two would leave SMs without work.
  const int qt = d <= 128 && items(2) >= n_sm ? 2 : 1;
  if (items(qt) > 0x7fffffffll) return FA2_ERR_INVALID_ARG;
  fa2::SeqMaps m;
  if (!map_packed(&m.q, Q, T, H, d, dtype, false, tpt, G) || !map_packed(&m.k, K, T, Hkv, d, dtype, true, 128, 1) ||
      !map_packed(&m.v, V, T, Hkv, d, dtype, true, 128, 1))
    return FA2_ERR_CUDA;
  fa2::SeqParams p = seq_params(O, LSE, cu_seqlens, st, B, T, H, Hkv, d, scale, causal, window);
  p.head_group = head_group(items(qt), 6, Hkv, n_sm);
  return fa2::launch_seq_packed(d, dtype == FA2_BF16, qt, m, p, dev, static_cast<unsigned int>(items(qt)),
                                reinterpret_cast<cudaStream_t>(stream));
}

size_t fa2_bwd_varlen_workspace_size(int B, int T, int H, int Hkv, int d) {
  if (check_sizes(B, T, H, Hkv, d, kMaxBwdHeadDim) != FA2_OK) return 0;
  const size_t rows = static_cast<size_t>(bwd_tiles(B, T, H / Hkv)) * Hkv * 128;
  const int split = bwd_split(B, T, Hkv);
  const size_t part = split > 1 ? static_cast<size_t>(split) * 2 * T * Hkv * bwd_tile_dim(d) * 4 : 0;
  return (2 * bwd_stat_bytes(B, T, H, Hkv) + rows * bwd_tile_dim(d) * 4 + part + 255) / 256 * 256;
}

int fa2_bwd_varlen(const fa2_packed* Q, const fa2_packed* K, const fa2_packed* V,
                   const fa2_packed* O, const fa2_packed* dO, const float* LSE,
                   const fa2_packed* dQ, const fa2_packed* dK, const fa2_packed* dV,
                   const int* cu_seqlens, void* workspace, size_t workspace_bytes, int B, int T,
                   int H, int Hkv, int d, float scale, int causal, int window, int dtype,
                   fa2_stream_t stream) {
  int rc = check_sizes(B, T, H, Hkv, d, kMaxBwdHeadDim);
  if (rc == FA2_OK) rc = check_mode(scale, causal, window, dtype);
  if (rc != FA2_OK) return rc;
  if (T == 0) return FA2_OK;
  for (const fa2_packed* x : {Q, O, dO, dQ})
    if (!packed_ok(x, T, H, d)) return FA2_ERR_INVALID_ARG;
  for (const fa2_packed* x : {K, V, dK, dV})
    if (!packed_ok(x, T, Hkv, d)) return FA2_ERR_INVALID_ARG;
  if (!LSE || !aligned(LSE, 4) || !cu_seqlens || !aligned(cu_seqlens, 4)) return FA2_ERR_INVALID_ARG;
  const void* all[9] = {dQ->data, dK->data, dV->data, Q->data, K->data, V->data, O->data, dO->data, LSE};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (all[i] == all[j]) return FA2_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < fa2_bwd_varlen_workspace_size(B, T, H, Hkv, d))
    return FA2_ERR_WORKSPACE;
  int dev, n_sm;
  unsigned int* st;
  rc = fa2::host_device(&dev, &n_sm, &st);
  if (rc != FA2_OK) return rc;
  const int G = H / Hkv, tpt = 128 / G, D = bwd_tile_dim(d);
  const long long tiles = bwd_tiles(B, T, G);
  const long long items = bwd_items(B, T, Hkv);
  if (tiles * 128 > 0x7fffffffll || items > (0x7fffffffll >> 3)) return FA2_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t stat = bwd_stat_bytes(B, T, H, Hkv);
  fa2::SeqBwdParams p{};
  p.O = static_cast<const uint16_t*>(O->data), p.o_row = O->stride_row, p.o_head = O->stride_head;
  p.dO = static_cast<const uint16_t*>(dO->data), p.do_row = dO->stride_row, p.do_head = dO->stride_head;
  p.dQ = static_cast<uint16_t*>(dQ->data), p.dq_row = dQ->stride_row, p.dq_head = dQ->stride_head;
  p.dK = static_cast<uint16_t*>(dK->data), p.dk_row = dK->stride_row, p.dk_head = dK->stride_head;
  p.dV = static_cast<uint16_t*>(dV->data), p.dv_row = dV->stride_row, p.dv_head = dV->stride_head;
  p.LSE = LSE;
  p.Dg = reinterpret_cast<float*>(ws);
  p.Lg = reinterpret_cast<float*>(ws + stat);
  p.acc = reinterpret_cast<float*>(ws + 2 * stat);
  p.kv_part = p.acc + static_cast<size_t>(tiles) * Hkv * 128 * D;
  p.split = bwd_split(B, T, Hkv);
  p.cu = cu_seqlens;
  p.status = st;
  p.wait_ns = fa2::host_wait_ns();
  p.fault = fa2::host_fault();
  p.B = B, p.T = T, p.Hkv = Hkv, p.G = G, p.d = d, p.tpt = tpt, p.tiles = static_cast<int>(tiles);
  p.causal = causal, p.window = std::min(window, T);  // no row sees more than T keys
  p.scale = scale, p.scale_log2 = scale * 1.4426950408889634f;
  p.head_group = head_group(items, 4, Hkv, n_sm);
  CUtensorMap m[5];
  const uint64_t adims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(tiles) * 128, static_cast<uint64_t>(Hkv)};
  const uint64_t astr[2] = {static_cast<uint64_t>(D) * 4, static_cast<uint64_t>(tiles) * 128 * D * 4};
  const uint32_t abox[3] = {32, 128, 1};
  if (!map_packed(&m[0], Q, T, H, d, dtype, false, tpt, G) || !map_packed(&m[1], K, T, Hkv, d, dtype, true, 128, 1) ||
      !map_packed(&m[2], V, T, Hkv, d, dtype, true, 128, 1) || !map_packed(&m[3], dO, T, H, d, dtype, false, tpt, G) ||
      !fa2::host_encode_map(&m[4], fa2::MapType::kF32, p.acc, 3, adims, astr, abox))
    return FA2_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned int n = static_cast<unsigned int>(items * p.split);
  return fa2::launch_seq_bwd(D, dtype == FA2_BF16, m, p, dev, n, s);
}

size_t fa2_fwd_paged_workspace_size(int B, int T, int H, int Hkv, int d, int sm_count) {
  if (check_sizes(B, T, H, Hkv, d, kMaxFwdHeadDim) != FA2_OK) return 0;
  if (sm_count <= 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        sm_count <= 0) {
      cudaGetLastError();
      return 0;
    }
  }
  return (paged_bytes(sm_count, form_tiles(paged_form(B, T, H / Hkv, d)), d) + 255) / 256 * 256;
}

int fa2_fwd_paged(const fa2_packed* Q, const fa2_cache* K, const fa2_cache* V, const fa2_packed* O,
                  float* LSE, const int* cu_seqlens, const int* seq_lens, const int* block_table,
                  void* workspace, size_t workspace_bytes, int B, int T, int H, int Hkv, int d,
                  int num_blocks, int block_size, int max_blocks, float scale, int causal,
                  int window, int dtype, fa2_stream_t stream) {
  int rc = check_sizes(B, T, H, Hkv, d, kMaxFwdHeadDim);
  if (rc == FA2_OK) rc = check_mode(scale, causal, window, dtype);
  if (rc != FA2_OK) return rc;
  if (num_blocks < 1 || max_blocks < 1 ||
      !(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64 ||
        (block_size >= 128 && block_size % 128 == 0)) ||
      static_cast<long long>(num_blocks) * block_size > 0x7fffffffll ||
      static_cast<long long>(max_blocks) * block_size > (1ll << 30))
    return FA2_ERR_INVALID_ARG;
  // Blocks of rows times key tiles times heads, which the kernel counts in 32 bits.  (The first
  // factors stay below 2^30 and 2^24.)
  const int G = H / Hkv, form = paged_form(B, T, G, d), tpt = form_tokens(form, G);
  const long long row_blocks = T / (tpt * form_tiles(form)) + static_cast<long long>(B);
  if (row_blocks * (static_cast<long long>(max_blocks) * block_size / 128 + 6) > (1ll << 30) / Hkv)
    return FA2_ERR_INVALID_ARG;
  if (T == 0) return FA2_OK;
  if (!packed_ok(Q, T, H, d) || !packed_ok(O, T, H, d) || !cache_ok(K, num_blocks, Hkv, block_size, d) ||
      !cache_ok(V, num_blocks, Hkv, block_size, d))
    return FA2_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(LSE), static_cast<const void*>(cu_seqlens),
                        static_cast<const void*>(seq_lens), static_cast<const void*>(block_table)})
    if (!x || !aligned(x, 4)) return FA2_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(Q->data), static_cast<const void*>(K->data),
                        static_cast<const void*>(V->data)})
    if (x == O->data || x == LSE) return FA2_ERR_INVALID_ARG;
  int dev, n_sm;
  unsigned int* st;
  rc = fa2::host_device(&dev, &n_sm, &st);
  if (rc != FA2_OK) return rc;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < fa2_fwd_paged_workspace_size(B, T, H, Hkv, d, n_sm))
    return FA2_ERR_WORKSPACE;
  fa2::SeqMaps m;
  if (!map_packed(&m.q, Q, T, H, d, dtype, false, tpt, G) ||
      !map_cache(&m.k, K, num_blocks, Hkv, block_size, d, dtype) ||
      !map_cache(&m.v, V, num_blocks, Hkv, block_size, d, dtype))
    return FA2_ERR_CUDA;
  fa2::SeqParams p = seq_params(O, LSE, cu_seqlens, st, B, T, H, Hkv, d, scale, causal, window);
  p.tpt = tpt;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.num_blocks = num_blocks, p.block_size = block_size, p.max_blocks = max_blocks;
  p.tiles_block = block_size / 128;
  for (p.box_shift = 3; 1 << p.box_shift < std::min(block_size, 128);) ++p.box_shift;
  p.O_part = static_cast<float*>(workspace);
  p.LSE_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + paged_opart_bytes(n_sm, form_tiles(form), d));
  p.merge = reinterpret_cast<int4*>(p.LSE_part + static_cast<size_t>(n_sm) * 2 * form_tiles(form) * 128);
  return fa2::launch_seq_paged(d, dtype == FA2_BF16, form, m, p, dev, static_cast<unsigned int>(n_sm),
                               reinterpret_cast<cudaStream_t>(stream));
}

int fa2_paged_tables(const int* context_lens, const int* new_lens, const int* free_blocks,
                     int num_free, int* block_table, int* cu_seqlens, int* seq_lens,
                     int* positions, int* slots, int* used, int B, int T, int block_size,
                     int max_blocks, fa2_stream_t stream) {
  if (B < 1 || T < 0 || num_free < 0 || block_size < 1 || max_blocks < 1 || B > (1 << 24) ||
      T > (1 << 30) || block_size > (1 << 20))
    return FA2_ERR_INVALID_ARG;
  const void* need[6] = {context_lens, new_lens, block_table, cu_seqlens, seq_lens, used};
  for (const void* x : need)
    if (!x || !aligned(x, 4)) return FA2_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_blocks) || (T > 0 && (!positions || !slots))) return FA2_ERR_INVALID_ARG;
  if (!aligned(free_blocks, 4) || !aligned(positions, 4) || !aligned(slots, 4)) return FA2_ERR_INVALID_ARG;
  int dev, n_sm;
  unsigned int* st;
  int rc = fa2::host_device(&dev, &n_sm, &st);
  if (rc != FA2_OK) return rc;
  fa2::TablesParams p{context_lens, new_lens, free_blocks, block_table, cu_seqlens, seq_lens, positions,
                      slots, used, num_free, B, T, block_size, max_blocks};
  const int grid = std::max(1, std::min(n_sm, (T + 2047) / 2048));
  fa2::fa2_paged_tables_kernel<<<grid, fa2::kTablesThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  fa2::host_count_launches(1);
  return FA2_OK;
}

int fa2_paged_append(const fa2_packed* K, const fa2_packed* V, const fa2_cache* K_cache,
                     const fa2_cache* V_cache, const int* slots, int T, int Hkv, int d,
                     int num_blocks, int block_size, fa2_stream_t stream) {
  int rc = check_sizes(1, T, Hkv, Hkv, d, kMaxFwdHeadDim);
  if (rc != FA2_OK) return rc;
  if (num_blocks < 1 || block_size < 1 ||
      static_cast<long long>(num_blocks) * block_size > 0x7fffffffll)
    return FA2_ERR_INVALID_ARG;
  if (T == 0) return FA2_OK;
  if (!packed_ok(K, T, Hkv, d) || !packed_ok(V, T, Hkv, d) ||
      !cache_ok(K_cache, num_blocks, Hkv, block_size, d) ||
      !cache_ok(V_cache, num_blocks, Hkv, block_size, d) || !slots || !aligned(slots, 4))
    return FA2_ERR_INVALID_ARG;
  const void* in[2] = {K->data, V->data};
  for (const void* x : in)
    if (x == K_cache->data || x == V_cache->data) return FA2_ERR_INVALID_ARG;
  if (K_cache->data == V_cache->data) return FA2_ERR_INVALID_ARG;
  int dev, n_sm;
  unsigned int* st;
  rc = fa2::host_device(&dev, &n_sm, &st);
  if (rc != FA2_OK) return rc;
  fa2::AppendParams p{};
  const fa2_packed* src[2] = {K, V};
  const fa2_cache* dst[2] = {K_cache, V_cache};
  for (int i = 0; i < 2; ++i) {
    p.src[i] = static_cast<const uint16_t*>(src[i]->data);
    p.dst[i] = static_cast<uint16_t*>(dst[i]->data);
    p.src_row[i] = src[i]->stride_row;
    p.src_head[i] = src[i]->stride_head;
    p.dst_block[i] = dst[i]->stride_block;
    p.dst_head[i] = dst[i]->stride_head;
    p.dst_row[i] = dst[i]->stride_row;
  }
  p.slots = slots;
  p.status = st;
  p.T = T, p.Hkv = Hkv, p.vec = d / 8, p.num_blocks = num_blocks, p.block_size = block_size;
  const int row = Hkv * p.vec, tx = std::min(row, fa2::kAppendThreads), ty = fa2::kAppendThreads / tx;
  const int per = fa2::kAppendRows * ty, pieces = (row + tx - 1) / tx;
  if (pieces > 32767) return FA2_ERR_INVALID_ARG;
  const dim3 grid((T + per - 1) / per, 2 * pieces);
  fa2::fa2_paged_append_kernel<<<grid, dim3(tx, ty), 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  fa2::host_count_launches(1);
  return FA2_OK;
}

}  // extern "C"
