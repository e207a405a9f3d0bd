// The packed forward kernels.
#include "fa2_seq_launch.cuh"

namespace fa2 {

int launch_seq_packed(int d, bool bf16, int qt, const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid,
                      cudaStream_t s) {
  return bf16 ? launch_seq_any<false, true>(d, qt, m, p, dev, grid, s) : launch_seq_any<false, false>(d, qt, m, p, dev, grid, s);
}

}  // namespace fa2
