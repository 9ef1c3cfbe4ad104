// csa2_decode.cuh -- cached entries and window tokens back to fp32, in units of
// eight values (exact: at most 8 significant bits times a power of two).
#pragma once

#include "csa2_device.cuh"

namespace csa2 {

__device__ __forceinline__ void e4m3x8(uint2 w, float s, float *v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e4m3_value(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu) * s;
}
__device__ __forceinline__ void bf16x8(uint4 w, float *v) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
// Unit u of window row `row` (a ring slot or a chunk's window row).
__device__ __forceinline__ void window_unit8(const uint8_t *codes, const uint8_t *scales, int swa_dtype, int64_t row,
                                             int u, float *v) {
  if (swa_dtype == CSA2_SWA_MXFP8)
    e4m3x8(reinterpret_cast<const uint2 *>(codes + row * 576)[u], e8m0_value(scales[row * kSwaScaleStride + (u >> 2)]), v);
  else
    bf16x8(reinterpret_cast<const uint4 *>(codes + row * 1152)[u], v);
}

}  // namespace csa2
