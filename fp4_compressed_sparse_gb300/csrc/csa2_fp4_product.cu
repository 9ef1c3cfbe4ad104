// csa2_fp4_product.cu -- out = x w^T of two 4-bit block-scaled matrices on the
// 5th-generation tensor cores (csa2_fp4_product).
//
// out[m][n] = r_m r_n sum_k x_mk w_nk: the block-scaled MMA multiplies E2M1 values and
// their block scales exactly and sums in fp32; the rows' powers of two are applied to
// the sum.  Operands lie in memory as the MMA reads them, so tiles go to shared memory
// by bulk copies and nothing is rearranged.
//
// k_fp4_split, up to 64 tokens or few tiles: the weights are the MMA's 128 rows (lane =
// output column, so a warp's stores are runs of one output row), the tokens its NT columns
// (all of them, or 128 at a time).  The K tiles of an output tile are dealt to the CTAs of a
// cluster, whose sums are added in rank order through distributed shared memory: no
// workspace, equal calls give equal bits.  Bound: the weights' bytes.  One token by 12,288 x
// 4,096 5.8 us with the weights in L2, 8.0 with each call's in HBM (28 MB: 3.5 TB/s, half the copy
// rate; no byte of them is requested before the kernel in front ends, and launch, tensor memory,
// first box and the join are 4.5 us of either), 501 tokens x 704 x 4,104 7.3.
//
// k_fp4_pair, more: 8,192 x 12,288 x 4,096 NV 121 us (6.8 PFLOP/s, 71 % of the 9.5 PFLOP/s
// that csa2_mxf4_peak_launch reaches), MX 113; 8,192^3 151 us (7.3).  Without its copies it
// takes 108 us, without its MMAs 105 (39 KB a stage and SM, 19 TB/s out of L2): two bounds
// that meet.  Tensor memory that never had to be drained would save 4 us.
#include <type_traits>

#include "csa2_fp4.cuh"
#include "csa2_tma.cuh"

namespace csa2 {
namespace {

constexpr uint32_t kWaitIters = 200;  // suspended polls of <= 1 ms each
constexpr int kSplitThreads = 192;    // producer, issuer, four epilogue warps

struct ProductArgs {
  csa2_fp4_matrix x, w;
  void *out;
  int64_t stride;
  int32_t *err;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// A map over a matrix's records, seen as [row tile][K tile][pieces][piece bytes], whose box
// is `pieces` pieces of k_tiles K tiles of row_tiles row tiles.
bool record_map(CUtensorMap *map, const csa2_fp4_matrix &m, bool nv, int pieces, int k_tiles, int row_tiles) {
  const uint64_t piece = nv ? 1024 : 512, rec = f4_tile_bytes(nv), kt = f4_col_tiles(m.cols);
  const uint64_t dim[4] = {piece / 8, rec / piece, kt, static_cast<uint64_t>(f4_row_tiles(m.rows))};
  const uint64_t stride[3] = {piece, rec, rec * kt};
  const uint32_t box[4] = {static_cast<uint32_t>(piece / 8), static_cast<uint32_t>(pieces), static_cast<uint32_t>(k_tiles),
                           static_cast<uint32_t>(row_tiles)};
  return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 4, m.tiles, dim, stride, box, false);
}
// A map over its codes, [row tile][K tile][32-column piece][row], whose box is the first nt
// rows of a tile in k_tiles K tiles.
bool token_map(CUtensorMap *map, const csa2_fp4_matrix &m, bool nv, int nt, int k_tiles) {
  const uint64_t rec = f4_tile_bytes(nv), kt = f4_col_tiles(m.cols);
  const uint64_t dim[4] = {2048 / 8, 4, kt, static_cast<uint64_t>(f4_row_tiles(m.rows))};
  const uint64_t stride[3] = {2048, rec, rec * kt};
  const uint32_t box[4] = {static_cast<uint32_t>(2 * nt), 4, static_cast<uint32_t>(k_tiles), 1};
  return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 4, m.tiles, dim, stride, box, false);
}
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(tc::smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}

// Shared memory of a stage, kTiles K tiles: the weights' records (128 rows), the tokens'
// codes and scales.  A copying thread takes about 0.2 us for a wait, an arming and a copy
// of any size, so a stage is as large as two CTAs per SM allow; with 128 tokens there is
// one per SM, and five stages (three: 501 x 704 x 4104 8.0 us against 7.2).
template <int NT, bool kNv>
struct Split {
  static constexpr int kTiles = NT <= 32 ? 4 : 2, kStages = NT <= 32 ? 2 : NT <= 64 ? 3 : 5;
  static constexpr int kRec = f4_tile_bytes(kNv), kS = f4_scale_bytes(kNv);
  static constexpr int kA = kTiles * kRec, kB = kTiles * NT * 64;
  static constexpr int kStage = kA + kB + kTiles * kS;
  static constexpr int kAtoms = kNv ? 2 : 1;    // 512 B of scales per operand and K tile
  static constexpr int kSfCols = 8 * kAtoms;    // TMEM columns of a K tile's scales
  static constexpr int kUsed = NT + kSfCols * kTiles * kStages, kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static constexpr int kPitch = 128 + 4;        // floats per token of the partial sums
  static constexpr int kBytes = (kStage * kStages > NT * kPitch * 4 ? kStage * kStages : NT * kPitch * 4) + 1024;
};

template <int n>
using Int = std::integral_constant<int, n>;

template <int NT, bool kNv, bool kBf16>
__global__ void __launch_bounds__(kSplitThreads)
    k_fp4_split(ProductArgs a, const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                const __grid_constant__ CUtensorMap ms) {
  using L = Split<NT, kNv>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t full[L::kStages], empty[L::kStages], done;
  __shared__ uint32_t tmem_at;
  __shared__ int loaded;  // stages whose copies were started
  __shared__ float r_tok[NT];
  __shared__ __align__(16) float r_col[kF4Rows];
  const uint32_t s0 = (tc::smem_addr(raw) + 1023) & ~1023u;
  uint8_t *smem = raw + (s0 - tc::smem_addr(raw));
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int nt = blockIdx.x / ranks, m0 = blockIdx.y * NT;
  const int kt = static_cast<int>(f4_col_tiles(a.x.cols)), steps = (kt + L::kTiles - 1) / L::kTiles;
  const int k0 = steps * static_cast<int>(rank) / static_cast<int>(ranks);
  const int nk = steps * static_cast<int>(rank + 1) / static_cast<int>(ranks) - k0;
  if (warp == 1) {
    tc::tmem_alloc(&tmem_at, L::kCols);
    tc::tmem_relinquish();
  }
  if (t == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    tc::mbar_init(&done, 1);
    loaded = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  next_may_start();
  wait_for_previous();
  const uint32_t tmem = tmem_at;

  if (warp >= 2) {  // the rows' powers of two, for the join (a load each there takes longer than the sums' way)
    const int i = t - 64;
    if (i < NT) r_tok[i] = m0 + i < a.x.rows ? a.x.row_scales[m0 + i] : 0.0f;
    r_col[i] = a.w.row_scales[nt * kF4Rows + i];  // (the plane holds whole tiles of rows)
  }
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < nk; ++i) {
      const int st = i % L::kStages;
      if (i >= L::kStages && !tc::mbar_wait_bounded(&empty[st], ((i / L::kStages) - 1) & 1, kWaitIters)) break;
      const uint32_t sa = s0 + st * L::kStage;
      const int k = (k0 + i) * L::kTiles;
      tc::mbar_expect_tx(&full[st], L::kStage);
      box_load(sa, &mw, 0, 0, k, nt, &full[st]);
      box_load(sa + L::kA, &mx, 0, 0, k, m0 / kF4Rows, &full[st]);
      box_load(sa + L::kA + L::kB, &ms, 0, kNv ? 8 : 16, k, m0 / kF4Rows, &full[st]);
      loaded = i + 1;
    }
  } else if (warp == 1) {
    const uint32_t el = elect_one();
    bool ok = true;
    for (int i = 0; i < nk && ok; ++i) {
      const int st = i % L::kStages;
      ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&full[st], (i / L::kStages) & 1, kWaitIters));
      if (!ok) break;
      tc::tc_fence_after();
      if (el) {
#pragma unroll
        for (int u = 0; u < L::kTiles; ++u) {
          const uint32_t sa = s0 + st * L::kStage + u * L::kRec, sb = s0 + st * L::kStage + L::kA + u * NT * 64;
          const uint32_t ss = s0 + st * L::kStage + L::kA + L::kB + u * L::kS;
          // a stage's scale columns are written again only once its MMAs, whose end
          // let the stage be refilled, are done
          const uint32_t sf = tmem + NT + (st * L::kTiles + u) * L::kSfCols;
#pragma unroll
          for (int h = 0; h < L::kAtoms; ++h) {
            tc::tmem_cp_32x128b_x4(sf + 4 * h, tc::smem_desc_noswizzle(sa + kF4CodeBytes + 512 * h, 128, 128));
            tc::tmem_cp_32x128b_x4(sf + 4 * (L::kAtoms + h), tc::smem_desc_noswizzle(ss + 512 * h, 128, 128));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tc::mma_f4<kNv>(tmem, tc::smem_desc_noswizzle(sa + 4096 * h, 2048, 128),
                            tc::smem_desc_noswizzle(sb + 2 * NT * 16 * h, NT * 16, 128), tc::idesc_f4(kNv, NT, kNv ? 0 : 2 * h),
                            sf + (kNv ? 4 * h : 0), sf + (kNv ? 8 + 4 * h : 4), i + u + h > 0 ? 1u : 0u);
        }
        tc::mma_commit(&empty[st]);
        if (i == nk - 1) tc::mma_commit(&done);
      }
      __syncwarp();
    }
  }
  __syncwarp();
  // every warp waits for the sums (each observes the phase itself)
  bool have = true;
  if (nk > 0) {
    int ok = 1;
    if (lane == 0) ok = tc::mbar_wait_bounded(&done, 0, kWaitIters) ? 1 : 0;
    have = __shfl_sync(0xffffffffu, ok, 0) != 0;
    if (have) tc::mbar_wait_bounded(&done, 0, kWaitIters);
    else if (lane == 0) raise_err(a.err, CSA2_DEVERR_TIMEOUT);
  }
  tc::tc_fence_after();
  // The block's vote: a wait may give up in one warp and just not in another, and all of them go the
  // same way here.  (After it the stages are free: every copy has landed, every MMA is done ...)
  have = __syncthreads_and(have);
  if (!have) {  // ... or a wait gave up: no copy may land later
    if (t == 0)
      for (int i = loaded > L::kStages ? loaded - L::kStages : 0; i < loaded; ++i)
        tc::mbar_wait_bounded(&full[i % L::kStages], (i / L::kStages) & 1, kWaitIters);
    __syncthreads();
  }
  float *part = reinterpret_cast<float *>(smem);
  if (warp >= 2) {
    const int q = warp & 3, n = 32 * q + lane;
#pragma unroll
    for (int c = 0; c < NT; c += 32) {
      uint32_t r[2][16];
      if (nk > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 16 * h < NT) tc::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * q) << 16) + c + 16 * h, r[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 16 * h < NT) tc::tmem_ld_wait_x16(r[h]);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < NT) part[(c + i) * L::kPitch + n] = nk > 0 ? __uint_as_float(r[i / 16][i % 16]) : 0.0f;
    }
  }
  tc::tc_fence_before();
  cluster_sync();
  // this CTA's share of the tokens: four columns a thread, the ranks' sums in order
  const int n_out = a.w.rows;
  const int per = (NT + ranks - 1) / ranks, c_lo = min(static_cast<int>(rank) * per, NT), c_hi = min(c_lo + per, NT);
  const int items = (min(c_hi, a.x.rows - m0) - c_lo) * 32;
  auto join = [&](auto held, auto most) {  // `held` at a time, all their loads in flight; up to `most` ranks
    constexpr int kH = decltype(held)::value, kR = decltype(most)::value;
    for (int i0 = t; i0 < items; i0 += kH * kSplitThreads) {
      float4 v[kH][kR];
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int i = i0 + h * kSplitThreads, c = c_lo + i / 32, n = 4 * (i % 32);
        if (i < items && nt * kF4Rows + n < n_out) {
#pragma unroll
          for (uint32_t k = 0; k < kR; ++k)
            if (k < ranks) v[h][k] = ld_cluster4(map_rank(tc::smem_addr(part + c * L::kPitch + n), k));
        }
      }
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int i = i0 + h * kSplitThreads, c = c_lo + i / 32, n = 4 * (i % 32), gn = nt * kF4Rows + n;
        if (i >= items || gn >= n_out) continue;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (uint32_t k = 0; k < kR; ++k)
          if (k < ranks) {
            s.x += v[h][k].x;
            s.y += v[h][k].y;
            s.z += v[h][k].z;
            s.w += v[h][k].w;
          }
        const float rm = r_tok[c];
        const float4 rn = *reinterpret_cast<const float4 *>(r_col + n);
        s.x *= rm * rn.x;
        s.y *= rm * rn.y;
        s.z *= rm * rn.z;
        s.w *= rm * rn.w;
        const int64_t at = (m0 + c) * a.stride + gn;
        if (gn + 4 <= n_out) {
          if constexpr (kBf16) {
            __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
                make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
          } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = s;
          }
        } else {
          const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (gn + j < n_out) {
              if constexpr (kBf16) static_cast<__nv_bfloat16 *>(a.out)[at + j] = __float2bfloat16_rn(o[j]);
              else static_cast<float *>(a.out)[at + j] = o[j];
            }
        }
      }
    }
  };
  if (ranks == 1) join(Int<8>{}, Int<1>{});
  else if (ranks <= 4) join(Int<4>{}, Int<4>{});
  else join(Int<2>{}, Int<8>{});
  cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, L::kCols);
  }
}

// ------------------------------------------------------------------ many tokens
// k_fp4_pair: persistent clusters of two CTAs, whose SMs' tensor cores work on one tile
// of 256 tokens x 256 columns (cta_group::2).  A CTA holds 128 of the tokens (and their
// sums, 256 columns of tensor memory) and the codes of 128 of the weights' rows; the
// scales of all 256 are needed by both.  The CTA of rank 0 issues for the two, and the
// copies of both signal its barriers.
//   warp 0      copies the tokens' records;  warp 2  the weights' codes;  warp 3  their scales
//   warp 1      (rank 0) scales to tensor memory, MMAs
//   warps 4-11  results: the sums are read into registers, which frees the tile's tensor
//               memory for the next one, then scaled and written
// (One CTA per tile of 128 x 256, its copies 2 KB pieces: 445 us for 8,192 x 12,288 x 4,096.)
// A stage is two K tiles (256 columns): a copying thread needs about 0.22 us for a wait,
// an arming and a copy, whatever its size.  Copies go by tensor maps over the records, so
// that one fetches a box of several records' codes or scales; what lies behind the last
// row or K tile arrives as zeros.
constexpr int kPairThreads = 384, kPairN = 256;
template <bool kNv>
struct Pair {
  static constexpr int kS = f4_scale_bytes(kNv), kRec = f4_tile_bytes(kNv), kAtoms = kNv ? 2 : 1;
  static constexpr int kA = 2 * kRec, kB = 2 * kF4CodeBytes, kStage = kA + kB + 4 * kS;
  static constexpr int kSfTile = kNv ? 24 : 16;  // TMEM columns of a K tile's scales: 8 per atom of the weights, then 4 per atom of the tokens
  static constexpr int kStages = kNv ? 5 : 6;
  static constexpr int kBytes = kStage * kStages + 1024;
};
constexpr int kPairStagesMax = 6;
struct PairSync {
  uint64_t full[kPairStagesMax], empty[kPairStagesMax];
  uint64_t tfull, tempty;
  uint32_t tmem;
  int loaded;  // stages rank 0 has armed
  int dead;    // a wait gave up
};

// Arrive on the barrier at the same place in CTA `rank` of the cluster.  Relaxed: what
// it hands over is tensor memory, which the tcgen05 fences on both sides order (a
// release at cluster scope takes a microsecond).
__device__ __forceinline__ void arrive_at(uint64_t *bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(map_rank(tc::smem_addr(bar), rank))
               : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                   tc::smem_addr(bar)),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}
// A box of the map to shared memory of this CTA; its bytes count on the barrier at
// (cluster) address bar, which may be the peer's.
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap *map, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(map), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(sdesc) : "memory");
}
template <bool kNv>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc) {
  if constexpr (kNv) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  }
}

__device__ __forceinline__ void put8(uint8_t *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void put4(uint8_t *p, const uint32_t *w) { *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]); }

template <bool kNv, bool kBf16>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_fp4_pair(ProductArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
               const __grid_constant__ CUtensorMap ms, int mt, int nt) {
  using L = Pair<kNv>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(128) PairSync sy;
  __shared__ __align__(16) float r_col[2][kPairN];  // powers of two of a tile's columns, and of the next one's
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int kt = static_cast<int>(f4_col_tiles(a.x.cols)), steps = (kt + 1) / 2;
  const int gm = (mt + 1) / 2, tiles = gm * nt, pairs = gridDim.x / 2;
  const uint32_t s0 = (tc::smem_addr(raw) + 1023) & ~1023u;  // (the same in both CTAs)
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(tc::smem_addr(&sy.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
  if (t == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(&sy.full[i], 1);
      tc::mbar_init(&sy.empty[i], 1);
    }
    tc::mbar_init(&sy.tfull, 1);
    tc::mbar_init(&sy.tempty, 16);
    sy.loaded = sy.dead = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised, its tensor memory allocated
  tc::tc_fence_after();
  next_may_start();
  wait_for_previous();
  const uint32_t tmem = sy.tmem;
  auto gave_up = [&]() {
    raise_err(a.err, CSA2_DEVERR_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sy.dead) = 1;
  };
  // tiles: down the tokens first, eight columns of tiles at a time
  auto tile_of = [&](int i, int &m, int &n) {
    constexpr int kBand = 8;
    const int band = i / (kBand * gm), in = i - band * kBand * gm, width = min(kBand, nt - band * kBand);
    m = 2 * (in / width) + static_cast<int>(rank);
    n = band * kBand + in % width;
  };
  const int first = blockIdx.x / 2;

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ copies
    const uint32_t el = elect_one();
    uint32_t st = 0, ph = 1;
    int f = 0;
    bool ok = true;
    for (int i = first; i < tiles && ok; i += pairs) {
      int m, n;
      tile_of(i, m, n);
      for (int k = 0; k < steps; ++k, ++f) {
        if (f >= L::kStages) ok = tc::mbar_wait_bounded(&sy.empty[st], ph, kWaitIters);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t sa = s0 + st * L::kStage, bar = map_rank(tc::smem_addr(&sy.full[st]), 0);
        if (el) {
          if (warp == 0) {
            if (rank == 0) tc::mbar_expect_tx(&sy.full[st], 2 * L::kStage);
            tensor_load(sa, &mx, 0, 2 * k, m, bar);
          } else if (warp == 2) {
            tensor_load(sa + L::kA, &mw, 0, 2 * k, 2 * n + static_cast<int>(rank), bar);
          } else {
            tensor_load(sa + L::kA + L::kB, &ms, kNv ? 8 : 16, 2 * k, 2 * n, bar);
          }
        }
        __syncwarp();
        if (++st == L::kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (t == 0 && rank == 0) sy.loaded = f;
    if (!ok && lane == 0) gave_up();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    const uint32_t el = elect_one();
    constexpr uint32_t kM256 = (128u >> 4) << 24;  // (the descriptor's M, from 128 to 256)
    constexpr uint32_t kId0 = tc::idesc_f4(kNv, kPairN, 0) + kM256, kId1 = tc::idesc_f4(kNv, kPairN, kNv ? 0 : 2) + kM256;
    uint32_t st = 0, ph = 0, j = 0;
    bool ok = true;
    for (int i = first; i < tiles && ok && rank == 0; i += pairs, ++j) {
      if (j > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&sy.tempty, (j - 1) & 1, kWaitIters));
      for (int k = 0; k < steps && ok; ++k) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&sy.full[st], ph, kWaitIters));
        if (!ok) break;
        tc::tc_fence_after();
        if (el) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t sa = s0 + st * L::kStage + u * L::kRec, sb = s0 + st * L::kStage + L::kA + u * kF4CodeBytes;
            const uint32_t ss = s0 + st * L::kStage + L::kA + L::kB + u * L::kS;  // columns 0-127; 128-255 two K tiles on
            const uint32_t sf = tmem + kPairN + (2 * st + u) * L::kSfTile;
            const uint64_t dsa = tc::smem_desc_noswizzle(sa + kF4CodeBytes, 128, 128), dsb = tc::smem_desc_noswizzle(ss, 128, 128),
                           da = tc::smem_desc_noswizzle(sa, 2048, 128), db = tc::smem_desc_noswizzle(sb, 2048, 128);
#pragma unroll
            for (int h = 0; h < L::kAtoms; ++h) {
              cp_scales_pair(sf + 8 * L::kAtoms + 4 * h, dsa + (512 * h >> 4));
              cp_scales_pair(sf + 8 * h, dsb + (512 * h >> 4));
              cp_scales_pair(sf + 8 * h + 4, dsb + ((2 * L::kS + 512 * h) >> 4));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_pair<kNv>(tmem, da + (4096 * h >> 4), db + (4096 * h >> 4), h ? kId1 : kId0,
                            sf + 8 * L::kAtoms + (kNv ? 4 * h : 0), sf + (kNv ? 8 * h : 0), k + u + h > 0 ? 1u : 0u);
          }
          commit_pair(&sy.empty[st]);
          if (k == steps - 1) commit_pair(&sy.tfull);
        }
        __syncwarp();
        if (++st == L::kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok && lane == 0) gave_up();
  } else {
    // ------------------------------------------------------------ results
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint32_t j = 0;
    bool gone = false;  // a wait gave up: the other warps still meet this one at the barrier
    for (int i = first; i < tiles; i += pairs, ++j) {
      int m, n;
      tile_of(i, m, n);
      const int row = m * kF4Rows + 32 * q + lane, c0 = n * kPairN + 128 * half;
      const bool live = row < a.x.rows;
      const float r_m = live ? a.x.row_scales[row] : 0.0f;
      const int col = n * kPairN + t - 128;  // (the row scales' plane holds whole tiles of 128)
      r_col[j & 1][t - 128] = col < static_cast<int>(f4_row_tiles(a.w.rows)) * kF4Rows ? a.w.row_scales[col] : 0.0f;
      __syncwarp();
      asm volatile("bar.sync 1, 256;\n" ::: "memory");  // warps 4-11
      const float *r_n = r_col[j & 1] + 128 * half;
      if (!gone) gone = !__all_sync(0xffffffffu, tc::mbar_wait_bounded(&sy.tfull, j & 1, kWaitIters));
      if (gone) continue;
      tc::tc_fence_after();
      uint32_t r[128];
      const uint32_t at = tmem + 128 * half + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll
      for (int c = 0; c < 8; ++c) tc::tmem_ld_32x32b_x16(at + 16 * c, r + 16 * c);
#pragma unroll
      for (int c = 0; c < 8; ++c) tc::tmem_ld_wait_x16(r + 16 * c);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(&sy.tempty, 0);
      const int cols = min(128, a.w.rows - c0);  // columns there are
      if (live && cols > 0) {
        // Whole sectors of 32 bytes a store (a lane's rows lie far apart: 16 bytes a store, fp32
        // 8,192 x 12,288 x 4,096 224 us against 156), from the second 16 bytes on where the row
        // begins in the middle of one.
        constexpr int kElt = kBf16 ? 2 : 4, kWords = 128 * kElt / 4, kStep = 32 * kElt / 4;
        uint8_t *p = static_cast<uint8_t *>(a.out) + (row * a.stride + c0) * kElt;
        const bool odd = reinterpret_cast<uintptr_t>(p) & 16;
        uint32_t w[kWords];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int c = 32 * k; c < 32 * k + 32; c += 4) {
            const float4 s = *reinterpret_cast<const float4 *>(r_n + c);
            const float v[4] = {__uint_as_float(r[c]) * (r_m * s.x), __uint_as_float(r[c + 1]) * (r_m * s.y),
                                __uint_as_float(r[c + 2]) * (r_m * s.z), __uint_as_float(r[c + 3]) * (r_m * s.w)};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if constexpr (!kBf16) w[c + u] = __float_as_uint(v[u]);
              else if (u % 2 == 0) {
                __nv_bfloat162 h = __floats2bfloat162_rn(v[u], v[u + 1]);
                w[(c + u) / 2] = *reinterpret_cast<uint32_t *>(&h);
              }
            }
          }
          const int at = kStep * k;  // words
          if (cols < 128) {          // the last columns: 16 bytes a store, then values
#pragma unroll
            for (int i = at; i < at + kStep; i += 4) {
              const int left = cols - i * 4 / kElt;
              if (left >= 16 / kElt) {
                put4(p + 4 * i, w + i);
              } else {
#pragma unroll
                for (int u = 0; u < 16 / kElt; ++u)
                  if (u < left) {
                    if constexpr (kBf16) reinterpret_cast<uint16_t *>(p + 4 * i)[u] = static_cast<uint16_t>(w[i + u / 2] >> (16 * (u & 1)));
                    else reinterpret_cast<uint32_t *>(p + 4 * i)[u] = w[i + u];
                  }
              }
            }
          } else if (odd) {
            if (k == 0) put4(p, w);
#pragma unroll
            for (int i = k ? at - 4 : 4; i + 8 <= at + kStep; i += 8) put8(p + 4 * i, w + i);
            if (k == 3) put4(p + 4 * (kWords - 4), w + kWords - 4);
          } else {
#pragma unroll
            for (int i = at; i < at + kStep; i += 8) put8(p + 4 * i, w + i);
          }
        }
      }
    }
    if (gone && lane == 0) gave_up();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (t == 0 && sy.dead)  // copies still in flight (rank 0: into either CTA)
    for (int i = sy.loaded > L::kStages ? sy.loaded - L::kStages : 0; i < sy.loaded; ++i)
      tc::mbar_wait_bounded(&sy.full[i % L::kStages], (i / L::kStages) & 1, kWaitIters);
  cluster_sync();  // neither leaves while the other's MMAs and arrivals may come
  if (warp == 1) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

template <bool kNv, bool kBf16>
cudaError_t launch_pair(const ProductArgs &a, cudaStream_t s) {
  using L = Pair<kNv>;
  const auto kern = k_fp4_pair<kNv, kBf16>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), L::kBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap mx, mw, ms;
  constexpr int kCodes = kNv ? 8 : 16;  // pieces of a record that are codes; one more is the scales
  if (!record_map(&mx, a.x, kNv, kCodes + 1, 2, 1) || !record_map(&mw, a.w, kNv, kCodes, 2, 1) || !record_map(&ms, a.w, kNv, 1, 2, 2))
    return cudaErrorNotSupported;
  const int mt = static_cast<int>(f4_row_tiles(a.x.rows)), nt = (a.w.rows + kPairN - 1) / kPairN;
  const int64_t tiles = static_cast<int64_t>((mt + 1) / 2) * nt, most = device_sm_count() / 2;
  return launch_after(kern, dim3(static_cast<unsigned>(2 * (tiles < most ? tiles : most))), kPairThreads, L::kBytes, 2, s, a, mx, mw, ms,
                      mt, nt);
}

template <int NT, bool kNv, bool kBf16>
cudaError_t launch_split(const ProductArgs &a, int ranks, cudaStream_t s) {
  using L = Split<NT, kNv>;
  const auto kern = k_fp4_split<NT, kNv, kBf16>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), L::kBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap mw, mx, ms;
  constexpr int kCodes = kNv ? 8 : 16;
  if (!record_map(&mw, a.w, kNv, kCodes + 1, L::kTiles, 1) || !token_map(&mx, a.x, kNv, NT, L::kTiles) ||
      !record_map(&ms, a.x, kNv, 1, L::kTiles, 1))
    return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(f4_row_tiles(a.w.rows) * ranks), static_cast<unsigned>((a.x.rows + NT - 1) / NT));
  return launch_after(kern, grid, kSplitThreads, L::kBytes, ranks, s, a, mw, mx, ms);
}
// Which kernel, and how the split one cuts the work.  One GB300, us, NV to bf16, in a graph.
//   Pairs for more than 64 tokens with more tiles of 128 x 128 than SMs (250 x 12288 x 512 6.0
//   against 11.3 split, x 4096 9.9 against 20.0), and with more than half as many if both CTAs of
//   a pair have tokens (250 x 9600 x 512 5.6 against 6.2, x 4096 9.5 against 10.7) or from 2,048
//   columns on (100 x 12288 x 4096 9.4 against 10.2, but x 1024 6.5 against 6.3), and of up to
//   1,024 columns from 32 tiles on (501 x 1024 x 512 5.2 against 5.8, 8,000 x 50 x 512 4.8 against
//   7.0); below, 250 x 4096 x 4096, of 64 tiles, 9.5 against 8.8.
//   Split: the narrowest token tile that holds all tokens, several tiles only of 128 (a tile of
//   64 that begins in the middle of a record would need that half's codes and, of the scales'
//   columns, those of rows 64 on, the last two of each four: not built), then as many ranks as are
//   resident at once, of 128 tokens one CTA per SM, else two: 64 x 12288 x 4096 8.1 with 3
//   against 12.1 with 1, 1 x 4096 x 8192 5.0 with 8 against 5.9 with 4, 501 x 704 x 4104 7.2 with
//   4 against 10.2 with 1.  Clusters do not cover all SMs: a few that wait for a second turn
//   cost as much as all (1 x 6144 x 4096 8.1 with 6, 4.9 with 4; 501 x 704 x 4104 10.8 with 6).
//   Of two stages none is dealt out (100 x 4096 x 512 6.2 with 2 ranks, 5.4 with 1).
// kRanks: ranks, the percentage of the SMs that clusters of so many cover with one CTA per
// SM (of 152: 152, 138, 144, 138, 120), and with two (of 304: 304, 291, 296, 276, 288).  Read
// from one GB300; where the SMs are spread otherwise over the GPU's clusters, a choice near
// its border can cost a second turn, and gives the same bits.
constexpr int kRanks[5][3] = {{2, 100, 100}, {3, 90, 95}, {4, 94, 97}, {6, 90, 90}, {8, 78, 95}};
template <bool kNv, bool kBf16>
cudaError_t launch_product(const ProductArgs &a, cudaStream_t s) {
  const int m = a.x.rows;
  const int64_t kt = f4_col_tiles(a.x.cols), sms = device_sm_count(), squares = f4_row_tiles(m) * f4_row_tiles(a.w.rows);
  const bool both = m > 128;
  if (m > 64 && (squares > sms || (2 * squares > sms && (both || kt >= 16)) || (both && kt <= 8 && squares >= 32)))
    return launch_pair<kNv, kBf16>(a, s);
  const int nt = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const int64_t tiles = f4_row_tiles(a.w.rows) * ((m + nt - 1) / nt), per = nt <= 32 ? 4 : 2, steps = (kt + per - 1) / per;
  int ranks = 1;
  for (const auto &r : kRanks)
    if (r[0] <= steps && steps > 2 && tiles * r[0] <= (nt < 128 ? 2 * sms * r[2] : sms * r[1]) / 100) ranks = r[0];
  switch (nt) {
    case 16: return launch_split<16, kNv, kBf16>(a, ranks, s);
    case 32: return launch_split<32, kNv, kBf16>(a, ranks, s);
    case 64: return launch_split<64, kNv, kBf16>(a, ranks, s);
    default: return launch_split<128, kNv, kBf16>(a, ranks, s);
  }
}

}  // namespace
}  // namespace csa2

extern "C" csa2_status csa2_fp4_product(const csa2_fp4_matrix *x, const csa2_fp4_matrix *w, void *out, int64_t out_stride,
                                        int32_t out_dtype, int32_t *err_word, csa2_stream_t stream) {
  csa2_status st = csa2::check_fp4(x, "x");
  if (st != CSA2_OK) return st;
  st = csa2::check_fp4(w, "w");
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(x->format == w->format, CSA2_ERR_RANGE, "formats %d and %d differ", x->format, w->format);
  CSA2_REQUIRE(x->cols == w->cols, CSA2_ERR_SHAPE, "x has %d columns, w %d", x->cols, w->cols);
  CSA2_REQUIRE(out_dtype == CSA2_OUT_F32 || out_dtype == CSA2_OUT_BF16, CSA2_ERR_RANGE, "out_dtype %d", out_dtype);
  CSA2_REQUIRE(out_stride >= w->rows && out_stride % 8 == 0, CSA2_ERR_SHAPE,
               "out_stride %lld must be a multiple of 8, %d at least", static_cast<long long>(out_stride), w->rows);
  if (x->rows == 0 || w->rows == 0) return CSA2_OK;
  CSA2_REQUIRE_PTR(out);
  const csa2::ProductArgs a{*x, *w, out, out_stride, err_word};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = out_dtype == CSA2_OUT_BF16;
  const cudaError_t e = x->format == CSA2_FP4_NV ? (bf ? csa2::launch_product<true, true>(a, s) : csa2::launch_product<true, false>(a, s))
                                                 : (bf ? csa2::launch_product<false, true>(a, s) : csa2::launch_product<false, false>(a, s));
  return csa2::cuda_status(e, "csa2_fp4_product launch");
}
