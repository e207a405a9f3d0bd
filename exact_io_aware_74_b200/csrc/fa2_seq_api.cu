// Host side of the packed-sequence and paged-cache entry points of libfa2.so:
// argument validation and launches.  Declarations and contracts are in include/fa2.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fa2.h"
#include "fa2_host.h"
#include "fa2_paged.cuh"
#include "fa2_varlen.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kMaxFwdHeadDim = 256;
constexpr int kMaxBwdHeadDim = 128;
constexpr int kMaxGroup = 128;  // query heads to a key/value head: rows of one query tile

int check_sizes(int B, int T, int H, int Hkv, int d, int max_d) {
  if (B < 1 || T < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > kMaxGroup) return FA2_ERR_INVALID_ARG;
  if (B > (1 << 24) || T > (1 << 30) || H > (1 << 16)) return FA2_ERR_INVALID_ARG;
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

fa2::Packed packed(const fa2_packed* x) {
  return {static_cast<uint16_t*>(x->data), x->stride_row, x->stride_head};
}
fa2::Cache cache(const fa2_cache* x) {
  return {static_cast<const uint16_t*>(x->data), x->stride_block, x->stride_head, x->stride_row};
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
  fa2::VarlenParams p{};
  p.Q = packed(Q);
  p.K = packed(K);
  p.V = packed(V);
  p.O = packed(O);
  p.LSE = LSE;
  p.cu = cu_seqlens;
  p.status = st;
  p.B = B, p.T = T, p.H = H, p.Hkv = Hkv, p.d = d, p.causal = causal, p.window = window;
  p.scale = scale;
  const dim3 grid((T + 3) / 4, H);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == FA2_BF16) fa2::fa2_varlen_fwd_plain<true, false><<<grid, 128, 0, s>>>(p);
  else fa2::fa2_varlen_fwd_plain<false, false><<<grid, 128, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  fa2::host_count_launches(1);
  return FA2_OK;
}

size_t fa2_bwd_varlen_workspace_size(int B, int T, int H, int Hkv, int d) {
  if (check_sizes(B, T, H, Hkv, d, kMaxBwdHeadDim) != FA2_OK) return 0;
  return (static_cast<size_t>(H) * T * 4 + 511) / 256 * 256;
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
  fa2::VarlenParams p{};
  p.Q = packed(Q);
  p.K = packed(K);
  p.V = packed(V);
  p.O = packed(O);
  p.dO = packed(dO);
  p.dQ = packed(dQ);
  p.dK = packed(dK);
  p.dV = packed(dV);
  p.LSE = const_cast<float*>(LSE);
  p.Dg = static_cast<float*>(workspace);
  p.cu = cu_seqlens;
  p.status = st;
  p.B = B, p.T = T, p.H = H, p.Hkv = Hkv, p.d = d, p.causal = causal, p.window = window;
  p.scale = scale;
  const dim3 gq((T + 3) / 4, H), gk((T + 3) / 4, Hkv);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == FA2_BF16) {
    fa2::fa2_varlen_dq_plain<true><<<gq, 128, 0, s>>>(p);
    fa2::fa2_varlen_dkv_plain<true><<<gk, 128, 0, s>>>(p);
  } else {
    fa2::fa2_varlen_dq_plain<false><<<gq, 128, 0, s>>>(p);
    fa2::fa2_varlen_dkv_plain<false><<<gk, 128, 0, s>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  fa2::host_count_launches(2);
  return FA2_OK;
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
  return 256;
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
  fa2::VarlenParams p{};
  p.Q = packed(Q);
  p.Kc = cache(K);
  p.Vc = cache(V);
  p.O = packed(O);
  p.LSE = LSE;
  p.cu = cu_seqlens;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.status = st;
  p.B = B, p.T = T, p.H = H, p.Hkv = Hkv, p.d = d, p.causal = causal, p.window = window;
  p.num_blocks = num_blocks, p.block_size = block_size, p.max_blocks = max_blocks;
  p.scale = scale;
  const dim3 grid((T + 3) / 4, H);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == FA2_BF16) fa2::fa2_varlen_fwd_plain<true, true><<<grid, 128, 0, s>>>(p);
  else fa2::fa2_varlen_fwd_plain<false, true><<<grid, 128, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  fa2::host_count_launches(1);
  return FA2_OK;
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
  const long long n = static_cast<long long>(T) * Hkv * p.vec;
  if ((n + 255) / 256 > 0x7fffffffll) return FA2_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned int>((n + 255) / 256), 2);
  fa2::fa2_paged_append_kernel<<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  fa2::host_count_launches(1);
  return FA2_OK;
}

}  // extern "C"
