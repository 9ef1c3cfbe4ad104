// csa2_ragged.cu -- writing a ragged batch's new tokens into the quantised cache
// (csa2_kv_append_ragged), and reading entries and the window back as the values
// they stand for (csa2_kv_read, csa2_window_read).
//
// The arithmetic is csa2_kv_append's (RoPE, then quantise; see csa2_encode.cuh),
// so the records are the same bytes.
//
// Bounds.  The append reads 1,408 B (bf16 rows) or 2,816 B (fp32) and a 256 B
// RoPE row per token and writes 392 B of records (724 B in the V4 format); the
// read moves the record and 2 or 4 B per value: both are bound by HBM at
// length, by launch and round trips for a few tokens.
#include "csa2_decode.cuh"
#include "csa2_encode.cuh"
#include "csa2_internal.cuh"

namespace csa2 {
namespace {

struct RaggedAppend {
  csa2_cache c;
  const void *kv, *ik;
  int64_t kv_stride, key_stride;
  int in_bf16;
  csa2_compress_in cmp;
  const int32_t *cu;
  int total, max_new;
  const float *rope_cs;
  int64_t rope_len;
  uint8_t *win_codes, *win_scales;  // the chunk's window rows, or nullptr
  int32_t *err;
};

__device__ __forceinline__ int swa_bytes(const csa2_cache &c) { return c.swa_dtype == CSA2_SWA_MXFP8 ? 576 : 1152; }

__device__ __forceinline__ float load_row(const void *p, int64_t i, int in_bf16) {
  if (in_bf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  return reinterpret_cast<const float *>(p)[i];
}

// Compression row `which` of token p of a sequence whose call rows start at
// `first` (token t0): the call's, or the compression buffer's for older tokens.
__device__ __forceinline__ const float *ragged_cmp_row(const RaggedAppend &a, int b, int first, int64_t t0, int64_t p,
                                                       int which) {
  if (p >= t0) {
    const float *src = which == 0 ? a.cmp.ca : which == 1 ? a.cmp.cb : which == 2 ? a.cmp.za : a.cmp.zb;
    return src + (first + (p - t0)) * kDcmp;
  }
  return a.c.cmp_buf + ((static_cast<size_t>(b) * 4 + (p & 3)) * 4 + which) * kDcmp;
}

// This block's part (row r of the call) of the compression buffer: token t's rows.
__device__ __forceinline__ void store_cmp_rows(const RaggedAppend &a, int b, int r, int64_t t) {
  float *dst = a.c.cmp_buf + (static_cast<size_t>(b) * 4 + (t & 3)) * 4 * kDcmp;
  const size_t src = static_cast<size_t>(r) * kDcmp;
  for (int i = threadIdx.x; i < kDcmp; i += blockDim.x) {
    dst[i] = a.cmp.ca[src + i];
    dst[kDcmp + i] = a.cmp.cb[src + i];
    dst[2 * kDcmp + i] = a.cmp.za[src + i];
    dst[3 * kDcmp + i] = a.cmp.zb[src + i];
  }
}

constexpr int kCopyBlocks = 4;  // blocks that copy one sequence's older window rows

// Blocks 0 .. total-1: one token each (entry, window row).  Further blocks: the
// 128 older window rows of each sequence.  single: max_new is 1 and there are
// no window rows to leave, so a token's block also finishes its sequence.
__global__ void __launch_bounds__(kEncThreads) k_ragged_append(RaggedAppend a, int single) {
  const csa2_cache &c = a.c;
  if (static_cast<int>(blockIdx.x) >= a.total) {
    const int part = blockIdx.x - a.total, b = part / kCopyBlocks, i0 = (part % kCopyBlocks) * (kWin / kCopyBlocks);
    int first, n;
    if (!ragged_rows(a.cu, b, a.total, a.max_new, first, n)) {
      if (i0 == 0 && threadIdx.x == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
      return;
    }
    const int64_t t0 = c.n_tokens[b] - kWin;
    const int row16 = swa_bytes(c) / 16;
    for (int k = threadIdx.x; k < kWin / kCopyBlocks * (row16 + 2); k += blockDim.x) {
      const int i = i0 + k / (row16 + 2), w = k % (row16 + 2);
      const int64_t t = t0 + i;
      const size_t dst = static_cast<size_t>(first) + static_cast<size_t>(kWin) * b + i;
      const size_t src = static_cast<size_t>(b) * kWin + (t & (kWin - 1));
      const uint4 zero = make_uint4(0, 0, 0, 0);
      if (w < row16)
        reinterpret_cast<uint4 *>(a.win_codes)[dst * row16 + w] =
            t >= 0 ? reinterpret_cast<const uint4 *>(c.swa_codes)[src * row16 + w] : zero;
      else if (c.swa_dtype == CSA2_SWA_MXFP8)
        reinterpret_cast<uint4 *>(a.win_scales)[dst * 2 + w - row16] =
            t >= 0 ? reinterpret_cast<const uint4 *>(c.swa_scales)[src * 2 + w - row16] : zero;
    }
    return;
  }
  __shared__ __align__(16) float row[kDcmp];
  __shared__ __align__(16) float rot[kRope];
  const int r = blockIdx.x;
  const int b = ragged_seq(a.cu, c.batch, r);
  if (b < 0) return;
  int first, n;
  if (!ragged_rows(a.cu, b, a.total, a.max_new, first, n)) {
    if (threadIdx.x == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
    return;
  }
  const int64_t t0 = c.n_tokens[b];
  if (!append_ok(c, t0, n, a.rope_len)) {
    if (r == first && threadIdx.x == 0) append_fail(c, t0, n, a.rope_len, a.err);
    return;
  }
  const int j = r - first;
  const int64_t t = t0 + j;
  const bool mine = c.ratio == 1;  // the entry is the token itself
  if (mine) {
    for (int i = threadIdx.x; i < kDqk; i += blockDim.x) row[i] = load_row(a.kv, r * a.kv_stride + i, a.in_bf16);
    for (int i = threadIdx.x; i < kDi; i += blockDim.x) row[kDqk + i] = load_row(a.ik, r * a.key_stride + i, a.in_bf16);
  } else {
    for (int i = threadIdx.x; i < kDqk; i += blockDim.x) row[i] = a.cmp.ca[static_cast<size_t>(r) * kDcmp + i];
  }
  if (threadIdx.x < 64) rot[threadIdx.x] = a.rope_cs[t * 64 + threadIdx.x];
  __syncthreads();
  block_rope_inplace(row, rot);
  __syncthreads();
  if (mine) block_encode_entry(c, b, t, row, rot, a.err);
  uint8_t *wc = nullptr, *ws = nullptr;
  if (a.win_codes != nullptr) {
    const size_t i = static_cast<size_t>(r) + static_cast<size_t>(kWin) * (b + 1);
    wc = a.win_codes + i * swa_bytes(c);
    ws = a.win_scales + i * kSwaScaleStride;
  } else if (j >= n - kWin) {
    const size_t i = static_cast<size_t>(b) * kWin + (t & (kWin - 1));
    wc = c.swa_codes + i * swa_bytes(c);
    ws = c.swa_scales + i * kSwaScaleStride;
  }
  if (wc != nullptr) block_encode_swa(wc, ws, c.swa_dtype, row, rot);
  if (!mine) {
    if (t & 1) {  // the pair is complete: entry t / 2, at position t - 1
      const int64_t e = t >> 1;
      const float *src[2][4];  // [Z, C][a0, a1, b0, b1]
      const bool has_b = e > 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t p = k < 2 ? 2 * e + k : has_b ? 2 * e - 4 + k : 2 * e;
        src[0][k] = ragged_cmp_row(a, b, first, t0, p, k < 2 ? 2 : 3);
        src[1][k] = ragged_cmp_row(a, b, first, t0, p, k < 2 ? 0 : 1);
      }
      __syncthreads();  // the window row has been read
      for (int i = threadIdx.x; i < kDcmp; i += blockDim.x)
        row[i] = r2_compress_channel(src[0][0][i], src[0][1][i], src[0][2][i], src[0][3][i], a.cmp.ba[i],
                                     a.cmp.ba[kDcmp + i], a.cmp.bb[i], a.cmp.bb[kDcmp + i], src[1][0][i], src[1][1][i],
                                     src[1][2][i], src[1][3][i], has_b);
      if (threadIdx.x < 64) rot[threadIdx.x] = a.rope_cs[(t - 1) * 64 + threadIdx.x];
      __syncthreads();
      block_rope_inplace(row, rot);
      __syncthreads();
      block_encode_entry(c, b, e, row, rot, a.err);
    }
    // a single token's slot (t % 4) is none of those its entry was made from
    if (single) store_cmp_rows(a, b, r, t);
  }
  if (single) {
    __syncthreads();  // every thread has read n_tokens
    if (threadIdx.x == 0) c.n_tokens[b] = t0 + n;
  }
}

// Once every token is encoded: the ring (from the window rows, when they were
// asked for), the compression buffer, n_tokens.  One block per sequence.
__global__ void __launch_bounds__(256) k_ragged_finish(RaggedAppend a) {
  const csa2_cache &c = a.c;
  const int b = blockIdx.x;
  int first, n;
  if (!ragged_rows(a.cu, b, a.total, a.max_new, first, n) || n == 0) return;
  const int64_t t0 = c.n_tokens[b];
  if (!append_ok(c, t0, n, a.rope_len)) return;
  if (a.win_codes != nullptr) {
    const int m = min(n, kWin), row16 = swa_bytes(c) / 16;
    const bool scales = c.swa_dtype == CSA2_SWA_MXFP8;
    for (int k = threadIdx.x; k < m * (row16 + 2); k += blockDim.x) {
      const int j = n - m + k / (row16 + 2), w = k % (row16 + 2);
      const size_t src = static_cast<size_t>(first) + j + static_cast<size_t>(kWin) * (b + 1);
      const size_t dst = static_cast<size_t>(b) * kWin + ((t0 + j) & (kWin - 1));
      if (w < row16)
        reinterpret_cast<uint4 *>(c.swa_codes)[dst * row16 + w] =
            reinterpret_cast<const uint4 *>(a.win_codes)[src * row16 + w];
      else if (scales)
        reinterpret_cast<uint4 *>(c.swa_scales)[dst * 2 + w - row16] =
            reinterpret_cast<const uint4 *>(a.win_scales)[src * 2 + w - row16];
    }
  }
  if (c.ratio == 2)
    for (int j = max(0, n - 4); j < n; ++j) store_cmp_rows(a, b, first + j, t0 + j);
  __syncthreads();
  if (threadIdx.x == 0) c.n_tokens[b] = t0 + n;
}

// ---------------------------------------------------------------- reading back
__device__ __forceinline__ void store8(void *out, int64_t at, int bf16, const float *v) {
  if (bf16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

struct ReadArgs {
  csa2_cache c;
  const int32_t *cu;
  int total;
  const int32_t *pos;
  const int64_t *start;
  void *main, *key;
  int64_t main_stride, key_stride;
  int bf16;
  int32_t *err;
};

// One warp per row, in units of 8 values: lane l has latent units l and l + 32,
// lanes 0-7 the RoPE units, lanes 8-23 the key's; every store instruction of
// the latent writes a contiguous 512 B (bf16).
__global__ void __launch_bounds__(256) k_kv_read(ReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= a.total) return;
  const csa2_cache &c = a.c;
  const int b = ragged_seq(a.cu, c.batch, r);
  if (b < 0) return;
  const int64_t e = a.pos ? static_cast<int64_t>(a.pos[r]) : a.start[b] + (r - a.cu[b]);
  int64_t pe = -1, pt = -1;
  bool bad = false;
  if (e >= 0) {
    const int64_t held = c.n_tokens[b] / c.ratio;
    bad = e >= held || e >= c.capacity;
    if (!bad) {
      const EntryMap map = entry_map(c);
      pe = phys_entry(map, b, e);
      pt = phys_tile(map, b, e / kIdxTile);
      bad = pe < 0 || pt < 0;
    }
  } else {
    bad = a.pos == nullptr;  // a negative start
  }
  if (bad && lane == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
  const bool some = e >= 0 && !bad;
  float v[8];
  auto zero = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  };
  if (a.main != nullptr) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = lane + 32 * k;
      zero();
      if (some) entry_unit8(c, pe, u, v);
      store8(a.main, r * a.main_stride + 8 * u, a.bf16, v);
    }
    if (lane < 8) {
      zero();
      if (some) entry_unit8(c, pe, 64 + lane, v);
      store8(a.main, r * a.main_stride + kLat + 8 * lane, a.bf16, v);
    }
  }
  if (a.key != nullptr && lane >= 8 && lane < 24) {
    const int u = lane - 8;
    zero();
    if (some) {
      const int m = static_cast<int>(e % kIdxTile);
      e2m1x8(*reinterpret_cast<const uint32_t *>(c.idx_codes + idx_code_at(pt, m, u >> 2) + 4 * (u & 3)),
             e8m0_value(c.idx_scales[idx_scale_at(pt, m) + (u >> 2)]), v);
    }
    store8(a.key, r * a.key_stride + 8 * u, a.bf16, v);
  }
}

// One thread per 8 values of a window token.
__global__ void __launch_bounds__(256) k_window_read(csa2_cache c, void *out, int bf16) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int u = static_cast<int>(id % (kDqk / 8));
  const int64_t at = id / (kDqk / 8);
  const int b = static_cast<int>(at / kWin), i = static_cast<int>(at % kWin);
  if (b >= c.batch) return;
  const int64_t t = c.n_tokens[b] - kWin + i;
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (t >= 0) {
    const size_t slot = static_cast<size_t>(b) * kWin + (t & (kWin - 1));
    window_unit8(c.swa_codes, c.swa_scales, c.swa_dtype, slot, u, v);
  }
  store8(out, at * kDqk + 8 * u, bf16, v);
}

}  // namespace
}  // namespace csa2

extern "C" {

using csa2::check_cache;
using csa2::cuda_status;

size_t csa2_chunk_window_bytes(int32_t batch, int32_t total, int32_t swa_dtype, int32_t plane) {
  if (batch <= 0 || total < 0) return 0;
  const size_t rows = static_cast<size_t>(total) + static_cast<size_t>(csa2::kWin) * batch;
  if (plane == 0) return rows * (swa_dtype == CSA2_SWA_MXFP8 ? 576 : 1152);
  return plane == 1 ? rows * csa2::kSwaScaleStride : 0;
}

csa2_status csa2_kv_append_ragged(const csa2_cache *cache, const void *kv, int64_t kv_stride, const void *idx_key,
                                  int64_t key_stride, int32_t in_dtype, const csa2_compress_in *cmp,
                                  const int32_t *cu_new, int32_t total, int32_t max_new, const float *rope_cs,
                                  int64_t rope_len, uint8_t *win_codes, uint8_t *win_scales, int32_t *err_word,
                                  csa2_stream_t stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(total >= 0 && total <= (1 << 24), CSA2_ERR_SHAPE, "total %d outside 0..2^24", total);
  CSA2_REQUIRE(max_new >= 0, CSA2_ERR_SHAPE, "max_new %d < 0", max_new);
  CSA2_REQUIRE_PTR(cu_new);
  CSA2_REQUIRE_PTR(rope_cs);
  CSA2_REQUIRE(rope_len >= 1, CSA2_ERR_SHAPE, "rope_len %lld < 1", static_cast<long long>(rope_len));
  if (cache->ratio == 1) {
    CSA2_REQUIRE(cmp == nullptr, CSA2_ERR_RANGE, "cmp must be NULL for a ratio-1 cache");
    CSA2_REQUIRE(in_dtype == CSA2_IN_F32 || in_dtype == CSA2_IN_BF16, CSA2_ERR_RANGE, "in_dtype %d", in_dtype);
    CSA2_REQUIRE_PTR(kv);
    CSA2_REQUIRE_PTR(idx_key);
    CSA2_REQUIRE(kv_stride >= CSA2_D_QK && kv_stride % 8 == 0, CSA2_ERR_SHAPE,
                 "kv_stride %lld must be a multiple of 8, 576 at least", static_cast<long long>(kv_stride));
    CSA2_REQUIRE(key_stride >= CSA2_D_INDEX && key_stride % 8 == 0, CSA2_ERR_SHAPE,
                 "key_stride %lld must be a multiple of 8, 128 at least", static_cast<long long>(key_stride));
  } else {
    CSA2_REQUIRE(cmp != nullptr, CSA2_ERR_NULL, "cmp is NULL for a ratio-2 cache");
    CSA2_REQUIRE_PTR(cmp->ca);
    CSA2_REQUIRE_PTR(cmp->cb);
    CSA2_REQUIRE_PTR(cmp->za);
    CSA2_REQUIRE_PTR(cmp->zb);
    CSA2_REQUIRE_PTR(cmp->ba);
    CSA2_REQUIRE_PTR(cmp->bb);
  }
  CSA2_REQUIRE_OPT_PTR(win_codes);
  CSA2_REQUIRE_OPT_PTR(win_scales);
  CSA2_REQUIRE(win_codes == nullptr || win_scales != nullptr || cache->swa_dtype == CSA2_SWA_BF16, CSA2_ERR_NULL,
               "win_scales is NULL for an MXFP8 window");
  if (total == 0 || max_new == 0) return CSA2_OK;
  csa2::RaggedAppend a{};
  a.c = *cache;
  a.kv = kv;
  a.ik = idx_key;
  a.kv_stride = kv_stride;
  a.key_stride = key_stride;
  a.in_bf16 = in_dtype == CSA2_IN_BF16;
  if (cmp != nullptr) a.cmp = *cmp;
  a.cu = cu_new;
  a.total = total;
  a.max_new = max_new;
  a.rope_cs = rope_cs;
  a.rope_len = rope_len;
  a.win_codes = win_codes;
  a.win_scales = win_scales;
  a.err = err_word;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int single = max_new == 1 && win_codes == nullptr;
  const int blocks = total + (win_codes != nullptr ? csa2::kCopyBlocks * cache->batch : 0);
  csa2::k_ragged_append<<<blocks, csa2::kEncThreads, 0, s>>>(a, single);
  if (!single) csa2::k_ragged_finish<<<cache->batch, 256, 0, s>>>(a);
  return cuda_status(cudaGetLastError(), "csa2_kv_append_ragged launch");
}

csa2_status csa2_kv_read(const csa2_cache *cache, const int32_t *cu_rows, int32_t total, const int32_t *pos,
                         const int64_t *start, void *out_main, int64_t main_stride, void *out_key, int64_t key_stride,
                         int32_t out_dtype, int32_t *err_word, csa2_stream_t stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(total >= 0 && total <= (1 << 30), CSA2_ERR_SHAPE, "total %d outside 0..2^30", total);
  CSA2_REQUIRE_PTR(cu_rows);
  CSA2_REQUIRE_OPT_PTR(pos);
  if (pos == nullptr) CSA2_REQUIRE_PTR(start);
  CSA2_REQUIRE(out_main != nullptr || out_key != nullptr, CSA2_ERR_NULL, "out_main and out_key are both NULL");
  CSA2_REQUIRE_OPT_PTR(out_main);
  CSA2_REQUIRE_OPT_PTR(out_key);
  CSA2_REQUIRE(out_dtype == CSA2_OUT_F32 || out_dtype == CSA2_OUT_BF16, CSA2_ERR_RANGE, "out_dtype %d", out_dtype);
  CSA2_REQUIRE(out_main == nullptr || (main_stride >= CSA2_D_QK && main_stride % 8 == 0), CSA2_ERR_SHAPE,
               "main_stride %lld must be a multiple of 8, 576 at least", static_cast<long long>(main_stride));
  CSA2_REQUIRE(out_key == nullptr || (key_stride >= CSA2_D_INDEX && key_stride % 8 == 0), CSA2_ERR_SHAPE,
               "key_stride %lld must be a multiple of 8, 128 at least", static_cast<long long>(key_stride));
  if (total == 0) return CSA2_OK;
  csa2::ReadArgs a{*cache, cu_rows, total, pos, start, out_main, out_key, main_stride, key_stride,
                   out_dtype == CSA2_OUT_BF16, err_word};
  csa2::k_kv_read<<<(total + 7) / 8, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError(), "csa2_kv_read launch");
}

csa2_status csa2_window_read(const csa2_cache *cache, void *out, int32_t out_dtype, csa2_stream_t stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE_PTR(out);
  CSA2_REQUIRE(out_dtype == CSA2_OUT_F32 || out_dtype == CSA2_OUT_BF16, CSA2_ERR_RANGE, "out_dtype %d", out_dtype);
  const int64_t units = static_cast<int64_t>(cache->batch) * csa2::kWin * (CSA2_D_QK / 8);
  csa2::k_window_read<<<static_cast<unsigned>((units + 255) / 256), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      *cache, out, out_dtype == CSA2_OUT_BF16);
  return cuda_status(cudaGetLastError(), "csa2_window_read launch");
}

}  // extern "C"
