// Launch of the forward kernels of fa2_seq_fwd.cuh; included by the unit that holds the
// packed kernels and the one that holds the paged kernels.
#pragma once

#include "../../include/fa2.h"
#include "fa2_host.h"
#include "fa2_seq_fwd.cuh"
#include "fa2_seq_host.h"

namespace fa2 {

template <int D, bool BF16, int QT, bool PAGED, int NQ = 0>
int launch_seq(const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid, cudaStream_t stream) {
  using Cfg = SeqCfg<D, QT, NQ>;
  auto kern = fa2_seq_fwd_kernel<D, BF16, QT, PAGED, NQ>;
  // The kernel re-splits its registers between warpgroups: only sound when every thread
  // was launched with exactly LAUNCH_REGS of them.
  static const bool regs_ok = [&] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess && fa.numRegs == Cfg::LAUNCH_REGS;
  }();
  static std::atomic<bool> smem_set[kSeqDevices];
  if (!regs_ok || !seq_smem_once(kern, dev, Cfg::SMEM, smem_set)) {
    cudaGetLastError();
    return FA2_ERR_CUDA;
  }
  kern<<<grid, Cfg::THREADS, Cfg::SMEM, stream>>>(m.q, m.k, m.v, p);
  if (cudaGetLastError() != cudaSuccess) return FA2_ERR_CUDA;
  host_count_launches(1);
  if constexpr (PAGED) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, NQ ? 1 : (QT == 1 ? 4 : 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fa2_seq_merge_kernel<D, BF16, QT>, p) != cudaSuccess) {
      cudaGetLastError();
      return FA2_ERR_CUDA;
    }
    host_count_launches(1);
  }
  return FA2_OK;
}

// form: 2 or 1 query tiles of 128 rows, or (paged, d <= 128) 16: few rows.
template <bool PAGED, bool BF16>
int launch_seq_any(int d, int form, const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid, cudaStream_t s) {
  if constexpr (PAGED) {
    if (form == 16) return d <= 64 ? launch_seq<64, BF16, 1, true, 16>(m, p, dev, grid, s) : launch_seq<128, BF16, 1, true, 16>(m, p, dev, grid, s);
  }
  switch (seq_tile_dim(d)) {
    case 64:
      return form == 2 ? launch_seq<64, BF16, 2, PAGED>(m, p, dev, grid, s) : launch_seq<64, BF16, 1, PAGED>(m, p, dev, grid, s);
    case 128:
      return form == 2 ? launch_seq<128, BF16, 2, PAGED>(m, p, dev, grid, s) : launch_seq<128, BF16, 1, PAGED>(m, p, dev, grid, s);
    case 192: return launch_seq<192, BF16, 1, PAGED>(m, p, dev, grid, s);
    default: return launch_seq<256, BF16, 1, PAGED>(m, p, dev, grid, s);
  }
}

}  // namespace fa2
