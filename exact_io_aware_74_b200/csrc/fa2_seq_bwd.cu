// The packed backward kernels.
#include "../../include/fa2.h"
#include "fa2_host.h"
#include "fa2_seq_bwd.cuh"
#include "fa2_seq_host.h"

namespace fa2 {

namespace {

template <typename... KArgs, typename... Args>
bool launch_chained(void (*kern)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  // Programmatic serialisation: the kernel may be set up while the one before it on the
  // stream finishes, and waits on the device before it reads.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) == cudaSuccess) {
    host_count_launches(1);
    return true;
  }
  cudaGetLastError();
  return false;
}

template <int D, bool BF16, bool SPLIT>
int launch_bwd_kernels(const CUtensorMap (&m)[5], const SeqBwdParams& p, int dev, unsigned int items, cudaStream_t s) {
  using Cfg = SeqBwdCfg<D>;
  auto kern = fa2_seq_bwd_kernel<D, BF16, SPLIT>;
  static std::atomic<bool> smem_set[kSeqDevices];
  if (!seq_smem_once(kern, dev, Cfg::SMEM, smem_set)) return FA2_ERR_CUDA;
  const dim3 rows(static_cast<unsigned int>(p.tiles) * (128 * D / 8 / 256), p.Hkv);
  if (!launch_chained(fa2_seq_bwd_pre_kernel<D, BF16>, rows, 256, 0, s, p) ||
      !launch_chained(kern, dim3(items), Cfg::THREADS, Cfg::SMEM, s, m[0], m[1], m[2], m[3], m[4], p) ||
      !launch_chained(fa2_seq_bwd_dq_kernel<D, BF16>, dim3(rows.x, p.split > 1 ? 2 * p.Hkv : p.Hkv), 256, 0, s, p))
    return FA2_ERR_CUDA;
  return FA2_OK;
}

template <int D, bool BF16>
int launch_split(const CUtensorMap (&m)[5], const SeqBwdParams& p, int dev, unsigned int items, cudaStream_t s) {
  return p.split > 1 ? launch_bwd_kernels<D, BF16, true>(m, p, dev, items, s)
                     : launch_bwd_kernels<D, BF16, false>(m, p, dev, items, s);
}

}  // namespace

int launch_seq_bwd(int D, bool bf16, const CUtensorMap (&m)[5], const SeqBwdParams& p, int dev, unsigned int items,
                   cudaStream_t s) {
  if (D == 64) return bf16 ? launch_split<64, true>(m, p, dev, items, s) : launch_split<64, false>(m, p, dev, items, s);
  return bf16 ? launch_split<128, true>(m, p, dev, items, s) : launch_split<128, false>(m, p, dev, items, s);
}

}  // namespace fa2
