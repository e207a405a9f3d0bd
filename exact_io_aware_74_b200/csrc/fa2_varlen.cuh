// Backward over packed sequences with grouped heads: plain kernels, one warp to a row,
// right for every size.
#pragma once

#include <cstdint>

#include "fa2_paged.cuh"
#include "ptx.cuh"

namespace fa2 {

struct Packed {
  uint16_t* data;
  long long row, head;
};

struct VarlenParams {
  Packed Q, K, V, O, dO, dQ, dK, dV;
  float* LSE;  // [H][T]
  float* Dg;   // [H][T]
  const int* cu;
  unsigned int* status;
  int B, T, H, Hkv, d, causal, window;
  float scale;
};

// Rows [start, start + len) of sequence b, clamped to the tensors.
__device__ __forceinline__ void seq_rows(const int* cu, int b, int T, int& start, int& len) {
  start = min(max(cu[b], 0), T);
  len = min(max(cu[b + 1], start), T) - start;
}

// The sequence that holds row t (-1: none): the last one that starts at or before t.
__device__ __forceinline__ int seq_of_row(const int* cu, int B, int T, int t) {
  int i = 0, j = B;
  while (j - i > 1) {
    const int m = (i + j) >> 1;
    if (cu[m] <= t) i = m; else j = m;
  }
  int s, n;
  seq_rows(cu, i, T, s, n);
  return (t >= s && t < s + n) ? i : -1;
}

template <bool BF16>
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  unpack2<BF16>(v.x, x[0], x[1]);
  unpack2<BF16>(v.y, x[2], x[3]);
  unpack2<BF16>(v.z, x[4], x[5]);
  unpack2<BF16>(v.w, x[6], x[7]);
}

template <bool BF16>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8], float f) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2<BF16>(x[0] * f, x[1] * f), pack2<BF16>(x[2] * f, x[3] * f),
                 pack2<BF16>(x[4] * f, x[5] * f), pack2<BF16>(x[6] * f, x[7] * f));
}

__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// dQ and D of a (row, query head).
template <bool BF16>
__global__ void __launch_bounds__(128) fa2_varlen_dq_plain(const VarlenParams p) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, lane = threadIdx.x & 31;
  if (t >= p.T) return;
  const int b = seq_of_row(p.cu, p.B, p.T, t);
  if (b < 0) return;
  int start, len;
  seq_rows(p.cu, b, p.T, start, len);
  const int i = t - start, hk = h / (p.H / p.Hkv);
  const int hi = p.causal ? i + 1 : len, lo = p.window > 0 ? max(0, i - p.window + 1) : 0;
  const bool on = lane * 8 < p.d;
  float q[8] = {}, o[8] = {}, g[8] = {}, acc[8] = {};
  if (on) {
    load8<BF16>(p.Q.data + t * p.Q.row + h * p.Q.head + lane * 8, q);
    load8<BF16>(p.O.data + t * p.O.row + h * p.O.head + lane * 8, o);
    load8<BF16>(p.dO.data + t * p.dO.row + h * p.dO.head + lane * 8, g);
  }
  const float D = dot8(o, g), L = p.LSE[static_cast<size_t>(h) * p.T + t];
  if (lane == 0) p.Dg[static_cast<size_t>(h) * p.T + t] = D;
  for (int j = lo; j < hi; ++j) {
    float k[8] = {}, v[8] = {};
    if (on) {
      load8<BF16>(p.K.data + (start + j) * p.K.row + hk * p.K.head + lane * 8, k);
      load8<BF16>(p.V.data + (start + j) * p.V.row + hk * p.V.head + lane * 8, v);
    }
    const float ds = expf(dot8(q, k) * p.scale - L) * (dot8(g, v) - D);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = fmaf(ds, k[c], acc[c]);
  }
  if (on) store8<BF16>(p.dQ.data + t * p.dQ.row + h * p.dQ.head + lane * 8, acc, p.scale);
}

// dK and dV of a (row, key/value head), summed over the query heads in order.
template <bool BF16>
__global__ void __launch_bounds__(128) fa2_varlen_dkv_plain(const VarlenParams p) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), hk = blockIdx.y, lane = threadIdx.x & 31;
  if (t >= p.T) return;
  const int b = seq_of_row(p.cu, p.B, p.T, t);
  if (b < 0) return;
  int start, len;
  seq_rows(p.cu, b, p.T, start, len);
  const int j = t - start, g = p.H / p.Hkv;
  const int lo = p.causal ? j : 0, hi = p.window > 0 ? min(len, j + p.window) : len;
  const bool on = lane * 8 < p.d;
  float k[8] = {}, v[8] = {}, dk[8] = {}, dv[8] = {};
  if (on) {
    load8<BF16>(p.K.data + t * p.K.row + hk * p.K.head + lane * 8, k);
    load8<BF16>(p.V.data + t * p.V.row + hk * p.V.head + lane * 8, v);
  }
  for (int h = hk * g; h < (hk + 1) * g; ++h)
    for (int i = lo; i < hi; ++i) {
      const int r = start + i;
      float q[8] = {}, dy[8] = {};
      if (on) {
        load8<BF16>(p.Q.data + r * p.Q.row + h * p.Q.head + lane * 8, q);
        load8<BF16>(p.dO.data + r * p.dO.row + h * p.dO.head + lane * 8, dy);
      }
      const size_t at = static_cast<size_t>(h) * p.T + r;
      const float w = expf(dot8(q, k) * p.scale - p.LSE[at]);
      const float ds = w * (dot8(dy, v) - p.Dg[at]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        dk[c] = fmaf(ds, q[c], dk[c]);
        dv[c] = fmaf(w, dy[c], dv[c]);
      }
    }
  if (on) {
    store8<BF16>(p.dK.data + t * p.dK.row + hk * p.dK.head + lane * 8, dk, p.scale);
    store8<BF16>(p.dV.data + t * p.dV.row + hk * p.dV.head + lane * 8, dv, 1.f);
  }
}

}  // namespace fa2
