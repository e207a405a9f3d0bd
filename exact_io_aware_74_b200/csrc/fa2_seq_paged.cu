// The paged forward kernels.
#include "fa2_seq_launch.cuh"

namespace fa2 {

int launch_seq_paged(int d, bool bf16, int form, const SeqMaps& m, const SeqParams& p, int dev, unsigned int grid,
                      cudaStream_t s) {
  return bf16 ? launch_seq_any<true, true>(d, form, m, p, dev, grid, s) : launch_seq_any<true, false>(d, form, m, p, dev, grid, s);
}

}  // namespace fa2
