// The paged forward kernels.
#include "fa2_seq_launch.cuh"

namespace fa2 {

int launch_seq_paged(int d, bool bf16, int qt, const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid,
                      cudaStream_t s) {
  return bf16 ? launch_seq_any<true, true>(d, qt, m, p, dev, grid, s) : launch_seq_any<true, false>(d, qt, m, p, dev, grid, s);
}

}  // namespace fa2
