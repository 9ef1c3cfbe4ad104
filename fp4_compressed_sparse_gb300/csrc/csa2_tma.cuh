// csa2_tma.cuh -- tensor maps for copies of boxes into shared memory.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace csa2 {

// A map over a tensor at `base` (16-byte aligned): dim[i] elements along dimension i
// (0 the innermost, contiguous), stride[i] bytes from one index of dimension i + 1 to the
// next (multiples of 16), box[i] of them a copy; 128-byte swizzle or none; indexes outside
// arrive as zeros.  False if the driver refuses it or has no such call.
bool tensor_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dim,
                const uint64_t *stride, const uint32_t *box, bool swizzle128);

}  // namespace csa2
