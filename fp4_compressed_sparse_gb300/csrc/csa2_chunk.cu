// csa2_chunk.cu -- dense attention of a ragged batch's new tokens over every
// visible cache entry and the sliding window (csa2_chunk_attn).
//
// z_j = sm_scale q . e_j over 576 dims, o = sum_j p_j c_j over the 512 latent
// dims, p the softmax with an optional sink in its denominator: one pass over
// the keys with a running maximum and sum in fp32.
//
// First form: one block per query token and 16 heads, fp32 FMAs on tiles of 16
// keys dequantised into shared memory.
#include <cmath>

#include "csa2_decode.cuh"
#include "csa2_internal.cuh"

namespace csa2 {
namespace {

struct ChunkArgs {
  csa2_cache c;
  const uint16_t *q;
  int heads;
  const int32_t *cu;
  int total, max_new;
  const uint8_t *win_codes, *win_scales;
  const float *sink;
  float sm_scale;
  void *out;
  int bf16;
  float *lse;
  int32_t *err;
};

constexpr int kHeadsPer = 16, kKeys = 16, kStride = kDqk + 4;

__global__ void __launch_bounds__(256) k_chunk_simple(ChunkArgs a) {
  extern __shared__ __align__(16) float sm[];
  float(*q)[kStride] = reinterpret_cast<float(*)[kStride]>(sm);
  float(*k)[kStride] = reinterpret_cast<float(*)[kStride]>(sm + kHeadsPer * kStride);
  __shared__ float p[kHeadsPer][kKeys + 1], m_s[kHeadsPer], l_s[kHeadsPer], al[kHeadsPer];
  __shared__ int live[kKeys];
  const int tid = threadIdx.x, r = blockIdx.x, h0 = blockIdx.y * kHeadsPer;
  const csa2_cache &c = a.c;
  const int b = ragged_seq(a.cu, c.batch, r);
  if (b < 0) return;
  int first, n;
  if (!ragged_rows(a.cu, b, a.total, a.max_new, first, n)) {
    if (tid == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
    return;
  }
  const int64_t ntok = c.n_tokens[b], pos = ntok - n + (r - first);
  int64_t T = pos > 0 ? pos / c.ratio : 0;
  if (T > c.capacity) T = c.capacity;
  for (int i = tid; i < kHeadsPer * kDqk; i += 256) {
    const int h = i / kDqk, d = i % kDqk;
    q[h][d] = __uint_as_float(static_cast<uint32_t>(a.q[(static_cast<size_t>(r) * a.heads + h0 + h) * kDqk + d]) << 16);
  }
  if (tid < kHeadsPer) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.0f;
  }
  float o[kHeadsPer][2] = {};
  const EntryMap map = entry_map(c);
  for (int64_t j0 = 0; j0 < T + kWin; j0 += kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * 72; i += 256) {
      const int kk = i / 72, u = i % 72;
      const int64_t j = j0 + kk;
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      int ok = 0;
      if (j < T) {
        const int64_t pe = phys_entry(map, b, j);
        if (pe >= 0) {
          entry_unit8(c, pe, u, v);
          ok = 1;
        } else {
          raise_err(a.err, CSA2_DEVERR_INDEX);
        }
      } else if (j < T + kWin) {
        const int64_t t = pos - (kWin - 1) + (j - T);
        if (t >= 0 && t <= pos) {
          if (a.win_codes != nullptr) {
            window_unit8(a.win_codes, a.win_scales, c.swa_dtype,
                         first + static_cast<int64_t>(kWin) * b + (t - (ntok - n - kWin)), u, v);
            ok = 1;
          } else if (t >= ntok - kWin) {
            window_unit8(c.swa_codes, c.swa_scales, c.swa_dtype, static_cast<int64_t>(b) * kWin + (t & (kWin - 1)), u, v);
            ok = 1;
          } else {
            raise_err(a.err, CSA2_DEVERR_INDEX);
          }
        }
      }
      if (u == 0) live[kk] = ok;
#pragma unroll
      for (int x = 0; x < 8; ++x) k[kk][8 * u + x] = v[x];
    }
    __syncthreads();
    {
      const int h = tid >> 4, kk = tid & 15;
      float s = 0.0f;
      for (int d = 0; d < kDqk; d += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(&q[h][d]), y = *reinterpret_cast<const float4 *>(&k[kk][d]);
        s = fmaf(x.x, y.x, s);
        s = fmaf(x.y, y.y, s);
        s = fmaf(x.z, y.z, s);
        s = fmaf(x.w, y.w, s);
      }
      s = live[kk] ? s * a.sm_scale : -INFINITY;
      float mx = s;
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float m_old = m_s[h], m_new = fmaxf(m_old, mx);
      const float e = m_new == -INFINITY ? 0.0f : expf(s - m_new);
      float sum = e;
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      p[h][kk] = e;
      __syncwarp();
      if (kk == 0) {
        al[h] = m_new == -INFINITY ? 1.0f : expf(m_old - m_new);
        l_s[h] = l_s[h] * al[h] + sum;
        m_s[h] = m_new;
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeadsPer; ++h) {
      o[h][0] *= al[h];
      o[h][1] *= al[h];
    }
    for (int kk = 0; kk < kKeys; ++kk) {
      const float2 v = *reinterpret_cast<const float2 *>(&k[kk][2 * tid]);
#pragma unroll
      for (int h = 0; h < kHeadsPer; ++h) {
        o[h][0] = fmaf(p[h][kk], v.x, o[h][0]);
        o[h][1] = fmaf(p[h][kk], v.y, o[h][1]);
      }
    }
  }
  __syncthreads();
  for (int h = 0; h < kHeadsPer; ++h) {
    float m = m_s[h], l = l_s[h], f = 1.0f;
    if (a.sink) {
      const float z = a.sink[h0 + h], mf = fmaxf(m, z);
      f = m == -INFINITY ? 0.0f : expf(m - mf);
      l = l * f + expf(z - mf);
      m = mf;
    }
    const float inv = l > 0.0f ? f / l : 0.0f;
    const size_t at = static_cast<size_t>(r) * a.heads + h0 + h;
    if (a.bf16)
      reinterpret_cast<__nv_bfloat162 *>(a.out)[at * (kLat / 2) + tid] = __floats2bfloat162_rn(o[h][0] * inv, o[h][1] * inv);
    else
      reinterpret_cast<float2 *>(a.out)[at * (kLat / 2) + tid] = make_float2(o[h][0] * inv, o[h][1] * inv);
    if (tid == 0) a.lse[at] = l > 0.0f ? m + logf(l) : -INFINITY;
  }
}

}  // namespace
}  // namespace csa2

extern "C" {

size_t csa2_chunk_attn_workspace_size(int32_t batch, int32_t total, int32_t n_heads) {
  (void)batch;
  (void)total;
  (void)n_heads;
  return 256;
}

csa2_status csa2_chunk_attn(const csa2_cache *cache, const uint16_t *q, int32_t n_heads, const int32_t *cu_q,
                            int32_t total, int32_t max_new, const uint8_t *win_codes, const uint8_t *win_scales,
                            const float *sink, float sm_scale, void *out, int32_t out_dtype, float *lse, void *ws,
                            size_t ws_bytes, int32_t *err_word, csa2_stream_t stream) {
  using csa2::cuda_status;
  csa2_status st = csa2::check_cache(cache);
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(total >= 0 && total <= (1 << 24), CSA2_ERR_SHAPE, "total %d outside 0..2^24", total);
  CSA2_REQUIRE(max_new >= 0, CSA2_ERR_SHAPE, "max_new %d < 0", max_new);
  CSA2_REQUIRE(n_heads >= 16 && n_heads <= CSA2_MAX_HEADS && n_heads % 16 == 0, CSA2_ERR_SHAPE,
               "n_heads %d must be a multiple of 16 in 16..128", n_heads);
  CSA2_REQUIRE_PTR(q);
  CSA2_REQUIRE_PTR(cu_q);
  CSA2_REQUIRE_OPT_PTR(win_codes);
  CSA2_REQUIRE_OPT_PTR(win_scales);
  CSA2_REQUIRE(win_codes == nullptr || win_scales != nullptr || cache->swa_dtype == CSA2_SWA_BF16, CSA2_ERR_NULL,
               "win_scales is NULL for an MXFP8 window");
  CSA2_REQUIRE_OPT_PTR(sink);
  CSA2_REQUIRE(std::isfinite(sm_scale), CSA2_ERR_RANGE, "sm_scale is not finite");
  CSA2_REQUIRE_PTR(out);
  CSA2_REQUIRE(out_dtype == CSA2_OUT_F32 || out_dtype == CSA2_OUT_BF16, CSA2_ERR_RANGE, "out_dtype %d", out_dtype);
  CSA2_REQUIRE_PTR(lse);
  const size_t need = csa2_chunk_attn_workspace_size(cache->batch, total, n_heads);
  CSA2_REQUIRE(ws != nullptr && ws_bytes >= need, CSA2_ERR_WORKSPACE, "chunk-attention workspace %zu < %zu bytes",
               ws_bytes, need);
  CSA2_REQUIRE(csa2::aligned16(ws), CSA2_ERR_ALIGN, "ws is not 16-byte aligned");
  if (total == 0 || max_new == 0) return CSA2_OK;
  csa2::ChunkArgs a{*cache, q, n_heads, cu_q, total, max_new, win_codes, win_scales, sink, sm_scale, out,
                    out_dtype == CSA2_OUT_BF16, lse, err_word};
  const int smem = (csa2::kHeadsPer + csa2::kKeys) * csa2::kStride * 4;
  cudaError_t e = csa2::ensure_smem_limit(reinterpret_cast<const void *>(&csa2::k_chunk_simple), smem);
  if (e != cudaSuccess) return cuda_status(e, "csa2_chunk_attn shared memory");
  csa2::k_chunk_simple<<<dim3(total, n_heads / csa2::kHeadsPer), 256, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError(), "csa2_chunk_attn launch");
}

}  // extern "C"
