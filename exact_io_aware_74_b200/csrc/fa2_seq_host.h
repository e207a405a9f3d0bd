// Launches of the packed and paged kernels, one translation unit each.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace fa2 {

struct SeqParams;

struct SeqMaps {
  CUtensorMap q, k, v;
};

// Kernel head dim (tile width) for head dim d.
inline int seq_tile_dim(int d) { return d <= 64 ? 64 : (d <= 128 ? 128 : (d <= 192 ? 192 : 256)); }

// qt: query tiles to an item, 1 or 2 (2 only up to d = 128).  form: 1 or 2 query tiles, or 16: items
// of at most 16 rows with the products' operands swapped (d <= 128).  grid: CTAs.  Both return an
// fa2_status.
int launch_seq_packed(int d, bool bf16, int qt, const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid,
                      cudaStream_t s);
int launch_seq_paged(int d, bool bf16, int form, const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid,
                     cudaStream_t s);

struct SeqBwdParams;

// D: tile width (64 or 128); maps: Q, K, V, dO, dQ accumulator.
int launch_seq_bwd(int D, bool bf16, const CUtensorMap (&maps)[5], const SeqBwdParams& p, int dev, unsigned int items,
                   cudaStream_t s);

// Raises a kernel's dynamic shared memory limit once per device; every kernel passes flags
// of its own.
constexpr int kSeqDevices = 64;
template <typename Kern>
bool seq_smem_once(Kern kern, int dev, int smem, std::atomic<bool> (&done)[kSeqDevices]) {
  if (dev < 0 || dev >= kSeqDevices) return false;
  if (done[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done[dev].store(true, std::memory_order_release);
  return true;
}

}  // namespace fa2
