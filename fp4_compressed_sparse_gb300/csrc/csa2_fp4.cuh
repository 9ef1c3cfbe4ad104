// csa2_fp4.cuh -- 4-bit block-scaled matrices: their layout and the tensor-core
// instructions that read it.
//
// A matrix of rows x cols is cut into tiles of 128 rows x 128 columns, row tile by
// row tile, each a record in the operand layout of the block-scaled MMA (K-major, no
// swizzle), so that it is copied into shared memory as it lies:
//   codes   j * 2048 + m * 16 + byte   (row m of the tile, 32-value piece j)
//   scales  behind them; NV (E4M3 per 16): h * 512 + 16 (m % 32) + 4 (m / 32) + g, group
//           4 h + g of the 8;  MX (E8M0 per 32): 16 (m % 32) + 4 (m / 32) + j
// and row_scales, fp32 per row.
#pragma once

#include "csa2_internal.cuh"
#include "csa2_tc.cuh"

namespace csa2 {

constexpr int kF4Rows = 128, kF4Cols = 128;
constexpr int kF4CodeBytes = 8192;  // of a tile
__host__ __device__ constexpr int f4_scale_bytes(bool nv) { return nv ? 1024 : 512; }
__host__ __device__ constexpr int f4_tile_bytes(bool nv) { return kF4CodeBytes + f4_scale_bytes(nv); }
__host__ __device__ __forceinline__ int64_t f4_col_tiles(int64_t cols) { return (cols + kF4Cols - 1) / kF4Cols; }
__host__ __device__ __forceinline__ int64_t f4_row_tiles(int64_t rows) { return (rows + kF4Rows - 1) / kF4Rows; }
// byte offset of the scale bytes of row m within a 512 B atom
__host__ __device__ __forceinline__ int f4_scale_at(int m) { return 16 * (m % 32) + 4 * (m / 32); }

namespace tc {

// Instruction descriptor of the block-scaled E2M1 kinds: K = 64, fp32 sums, both
// operands K-major; UE4M3 scales (4 per 64) or UE8M0 (2 per 64, sf selects the pair).
__host__ __device__ constexpr uint32_t idesc_f4(bool nv, int N, int sf) {
  return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         ((nv ? 0u : 1u) << 23) | (static_cast<uint32_t>(128 >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}
template <bool kNv>
__device__ __forceinline__ void mma_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t acc) {
  if constexpr (kNv) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  } else {
    mma_mxf4(d, a, b, idesc, sfa, sfb, acc);
  }
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

}  // namespace tc
}  // namespace csa2
