// Host services of fa2_api.cu that the other translation units of the library use.
#pragma once

#include <cstdint>

#include <cuda.h>

namespace fa2 {

// Checks that the current device is a B200 and returns its ordinal, its SM count and
// the library's status word there; FA2_OK or an fa2_status.
int host_device(int* dev, int* n_sm, unsigned int** status);

// Budget of one bounded in-kernel wait, the fault-injection hook, and the launch count.
unsigned long long host_wait_ns();
int host_fault();
void host_count_launches(unsigned long long n);

// cuTensorMapEncodeTiled with 128-byte swizzle, zero fill and unit element strides;
// dims, strides (bytes, rank - 1 of them) and box innermost first.  False on failure.
enum class MapType { kF16, kBF16, kF32 };
bool host_encode_map(CUtensorMap* map, MapType type, const void* base, int rank, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box);

}  // namespace fa2
