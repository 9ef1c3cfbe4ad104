// csa2_fp4_product.cu -- out = x w^T of two 4-bit block-scaled matrices on the
// 5th-generation tensor cores (csa2_fp4_product).
//
// out[m][n] = r_m r_n sum_k x_mk w_nk: the block-scaled MMA multiplies E2M1 values and
// their block scales exactly and sums in fp32; the rows' powers of two are applied to
// the sum.  Operands lie in memory as the MMA reads them, so tiles go to shared memory
// by bulk copies and nothing is rearranged.
//
// k_fp4_split: the weights are the MMA's 128 rows (lane = output column, so a warp's
// stores are runs of one output row), the tokens its NT columns.  The K tiles of an
// output tile are dealt to the CTAs of a cluster, whose sums are added in rank order
// through distributed shared memory: no workspace, equal calls give equal bits.
// Bound: the weights' bytes for few tokens.
#include "csa2_fp4.cuh"

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

// Shared memory of a stage: codes of 128 weight rows, codes of NT tokens, both's scales.
template <int NT, bool kNv>
struct Split {
  static constexpr int kA = kF4TileBytes, kB = NT * 64, kS = f4_scale_tile(kNv);
  static constexpr int kStage = kA + kB + 2 * kS;
  static constexpr int kStages = NT <= 32 ? 8 : NT <= 64 ? 7 : 5;  // two CTAs per SM
  static constexpr int kAtoms = kNv ? 2 : 1;                       // 512 B of scales per operand
  static constexpr int kSfCols = 8 * kAtoms;                       // TMEM columns of a stage's scales
  static constexpr int kCols = NT + kSfCols * kStages <= 128 ? 128 : 256;
  static constexpr int kPitch = 128 + 4;                           // floats per token of the partial sums
  static constexpr int kBytes = kStage * kStages > NT * kPitch * 4 ? kStage * kStages : NT * kPitch * 4;
};

template <int NT, bool kNv, bool kBf16>
__global__ void __launch_bounds__(kSplitThreads) k_fp4_split(ProductArgs a) {
  using L = Split<NT, kNv>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[L::kStages], empty[L::kStages], done;
  __shared__ uint32_t tmem_at;
  __shared__ int loaded;  // K tiles whose copies were started
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int nt = blockIdx.x / ranks, m0 = blockIdx.y * NT;
  const int kt = static_cast<int>(f4_col_tiles(a.x.cols));
  const int k0 = kt * static_cast<int>(rank) / static_cast<int>(ranks), k1 = kt * static_cast<int>(rank + 1) / static_cast<int>(ranks);
  const int nk = k1 - k0;
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
  const uint32_t tmem = tmem_at, s0 = tc::smem_addr(smem);

  if (warp == 0 && lane == 0) {
    const int64_t wt = static_cast<int64_t>(nt) * kt, xt = static_cast<int64_t>(m0 / kF4Rows) * kt;
    for (int i = 0; i < nk; ++i) {
      const int st = i % L::kStages;
      if (i >= L::kStages && !tc::mbar_wait_bounded(&empty[st], ((i / L::kStages) - 1) & 1, kWaitIters)) break;
      const uint32_t sa = s0 + st * L::kStage, sb = sa + L::kA, ss = sb + L::kB;
      tc::mbar_expect_tx(&full[st], L::kStage);
      tc::bulk_load(sa, a.w.codes + (wt + k0 + i) * kF4TileBytes, L::kA, &full[st]);
      const uint8_t *xc = a.x.codes + (xt + k0 + i) * kF4TileBytes;
      if constexpr (NT == 128) {
        tc::bulk_load(sb, xc, L::kB, &full[st]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) tc::bulk_load(sb + j * NT * 16, xc + j * 2048, NT * 16, &full[st]);
      }
      tc::bulk_load(ss, a.w.scales + (wt + k0 + i) * L::kS, L::kS, &full[st]);
      tc::bulk_load(ss + L::kS, a.x.scales + (xt + k0 + i) * L::kS, L::kS, &full[st]);
      loaded = i + 1;
    }
  } else if (warp == 1 && lane == 0) {
    bool ok = true;
    for (int i = 0; i < nk && ok; ++i) {
      const int st = i % L::kStages;
      ok = tc::mbar_wait_bounded(&full[st], (i / L::kStages) & 1, kWaitIters);
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t sa = s0 + st * L::kStage, sb = sa + L::kA, ss = sb + L::kB;
      // a stage's scale columns are written again only once its MMAs, whose end
      // let the stage be refilled, are done
      const uint32_t sf = tmem + NT + st * L::kSfCols;
#pragma unroll
      for (int h = 0; h < L::kAtoms; ++h) {
        tc::tmem_cp_32x128b_x4(sf + 4 * h, tc::smem_desc_noswizzle(ss + 512 * h, 128, 128));
        tc::tmem_cp_32x128b_x4(sf + 4 * (L::kAtoms + h), tc::smem_desc_noswizzle(ss + L::kS + 512 * h, 128, 128));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sfa = sf + (kNv ? 4 * h : 0), sfb = sf + (kNv ? 8 + 4 * h : 4);
        tc::mma_f4<kNv>(tmem, tc::smem_desc_noswizzle(sa + 4096 * h, 2048, 128),
                        tc::smem_desc_noswizzle(sb + 2 * NT * 16 * h, NT * 16, 128), tc::idesc_f4(kNv, NT, kNv ? 0 : 2 * h), sfa,
                        sfb, i + h > 0 ? 1u : 0u);
      }
      tc::mma_commit(&empty[st]);
    }
    if (ok) tc::mma_commit(&done);
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
  __syncthreads();  // (the stages are free: every copy has landed, every MMA is done)
  if (!have) {      // ... or a wait gave up: no copy may land later
    if (t == 0)
      for (int i = loaded > L::kStages ? loaded - L::kStages : 0; i < loaded; ++i)
        tc::mbar_wait_bounded(&full[i % L::kStages], (i / L::kStages) & 1, kWaitIters);
    __syncthreads();
  }
  float *part = reinterpret_cast<float *>(smem);
  if (warp >= 2) {
    const int q = warp & 3, n = 32 * q + lane;
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      uint32_t r[16];
      if (nk > 0) {
        tc::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * q) << 16) + c, r);
        tc::tmem_ld_wait_x16(r);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c + i) * L::kPitch + n] = nk > 0 ? __uint_as_float(r[i]) : 0.0f;
    }
  }
  tc::tc_fence_before();
  cluster_sync();
  // this CTA's share of the tokens: four columns a thread, the ranks' sums in order
  const int n_out = a.w.rows;
  const int per = (NT + ranks - 1) / ranks, c_lo = min(static_cast<int>(rank) * per, NT), c_hi = min(c_lo + per, NT);
  for (int i = t; i < (c_hi - c_lo) * 32; i += kSplitThreads) {
    const int c = c_lo + i / 32, n = 4 * (i % 32), m = m0 + c, gn = nt * kF4Rows + n;
    if (m >= a.x.rows || gn >= n_out) continue;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (uint32_t k = 0; k < ranks; ++k) {
      const float4 v = ld_cluster4(map_rank(tc::smem_addr(part + c * L::kPitch + n), k));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float rm = a.x.row_scales[m];
    const float4 rn = *reinterpret_cast<const float4 *>(a.w.row_scales + gn);  // (the plane holds whole tiles of rows)
    s.x *= rm * rn.x;
    s.y *= rm * rn.y;
    s.z *= rm * rn.z;
    s.w *= rm * rn.w;
    const int64_t at = m * a.stride + gn;
    if (gn + 4 <= n_out) {
      if constexpr (kBf16) {
        __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
            make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
      } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = s;
      }
    } else {
      const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (gn + j < n_out) {
          if constexpr (kBf16) static_cast<__nv_bfloat16 *>(a.out)[at + j] = __float2bfloat16_rn(v[j]);
          else static_cast<float *>(a.out)[at + j] = v[j];
        }
    }
  }
  cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, L::kCols);
  }
}

template <int NT, bool kNv, bool kBf16>
cudaError_t launch_split(const ProductArgs &a, int ranks, cudaStream_t s) {
  using L = Split<NT, kNv>;
  const void *fn = reinterpret_cast<const void *>(k_fp4_split<NT, kNv, kBf16>);
  cudaError_t e = ensure_smem_limit(fn, L::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(f4_row_tiles(a.w.rows) * ranks), static_cast<unsigned>((a.x.rows + NT - 1) / NT));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_fp4_split<NT, kNv, kBf16>, a);
}
template <bool kNv, bool kBf16>
cudaError_t launch_product(const ProductArgs &a, cudaStream_t s) {
  const int m = a.x.rows;
  const int nt = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const int64_t tiles = f4_row_tiles(a.w.rows) * ((m + nt - 1) / nt);
  const int64_t kt = f4_col_tiles(a.x.cols), sms = device_sm_count();
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= 2 * sms && kt >= 4 * ranks) ranks *= 2;
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
