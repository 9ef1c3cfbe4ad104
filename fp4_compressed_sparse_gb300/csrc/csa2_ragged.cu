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
  csa2_compress_in cmp;
  const int32_t *cu;
  int total, max_new;
  const float *rope_cs;
  int64_t rope_len;
  uint8_t *win_codes, *win_scales;  // the chunk's window rows, or nullptr
  int32_t *err;
};

__device__ __forceinline__ int swa_bytes(const csa2_cache &c) { return c.swa_dtype == CSA2_SWA_MXFP8 ? 576 : 1152; }

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

// Part `part` of the window rows of the tokens before the chunk.
__device__ __forceinline__ void copy_older(const RaggedAppend &a, int part) {
  const csa2_cache &c = a.c;
  const int b = part / kCopyBlocks, i0 = (part % kCopyBlocks) * (kWin / kCopyBlocks);
  int first, n;
  if (!ragged_rows(a.cu, b, a.total, a.max_new, first, n)) {
    if (i0 == 0 && threadIdx.x == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
    return;
  }
  if (!block_ragged_own(a.cu, c.batch, b, first, n)) return;  // (where the list decreases, the bit is raised)
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
}

// Sequences without a row of theirs in the arrays are nobody's to report: a call
// whose tokens' blocks are its only ones has some more for the list itself.
__device__ __forceinline__ void check_list(const RaggedAppend &a, int part) {
  const int b = part * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
  int first, n;
  if (b < a.c.batch && !ragged_rows(a.cu, b, a.total, a.max_new, first, n)) raise_err(a.err, CSA2_DEVERR_INDEX);
}

// ---------------------------------------------------------------- ratio 1: a warp per token
// Lane l has latent dims 16 l .. + 15 (one NVFP4 group, half an MXFP8 block), RoPE
// pair l, key dims 4 l .. + 3, all in registers: no shared memory, no barrier.  While
// the row is on its way the warp finds where it goes (a chain of dependent loads:
// the sequence, its length, the page).
//
// 32,768 bf16 tokens in the V4 format take 24 us: 70 MB, 2.9 TB/s, 43 % of the
// measured HBM rate; 12,871 fp32 tokens in FP4 19.5 us.  Nothing is saturated (SM
// 59 %, ALU 53 %, DRAM 27 %): the quantisers' instructions and the round trips share
// the time.  Latency is hidden by other warps, four blocks per SM (64 registers).  One thread per token finding its place for
// the block, with a barrier, took 27 us; several tokens per warp, the next row
// requested ahead, 30 us; a block per token through shared memory 261 us.

// Sixteen E2M1 codes of x / s without the divisions: x / s, rounded to fp32, is at
// most (below) a midpoint t of the grid exactly when x is at most (below) t s.
// t s is exact (3 + 4 significant bits), and the next fp32 number from t s differs
// by at least 2^-24 of it, the rounding of the quotient next to t by no more than
// 2^-24 of t: never enough to carry it over (2^-25 below a power of two).
__device__ __forceinline__ uint2 nvfp4_16(const float *x, uint32_t *scale) {
  float amax = fabsf(x[0]);  // (NaN only where all sixteen are)
#pragma unroll
  for (int i = 1; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  const uint32_t sc = e4m3_code(__fdiv_rn(amax, 6.0f));
  const float s = e4m3_value(sc);
  if (s == 0.0f) {
    *scale = 0;
    return make_uint2(0, 0);
  }
  *scale = sc;
  // (the sign bit of x s is that of x / s, which loses a NaN's)
  // |x| >= T[i] <=> code > i; ties go to the even code, so every other bound is
  // the number after the midpoint
  const uint32_t T0 = __float_as_uint(0.25f * s) + 1, T1 = __float_as_uint(0.75f * s), T2 = __float_as_uint(1.25f * s) + 1,
                 T3 = __float_as_uint(1.75f * s), T4 = __float_as_uint(2.5f * s) + 1, T5 = __float_as_uint(3.5f * s),
                 T6 = __float_as_uint(5.0f * s) + 1;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t v = __float_as_uint(x[i]) & 0x7FFFFFFFu, u = __float_as_uint(__fmul_rn(x[i], s));
    const bool g4 = v >= T3, g2 = v >= (g4 ? T5 : T1);
    const bool g1 = v >= (g4 ? (g2 ? T6 : T4) : (g2 ? T2 : T0));
    const uint32_t code = (g4 ? 4u : 0u) | (g2 ? 2u : 0u) | (g1 ? 1u : 0u) | ((u >> 28) & 8u);
    w[i / 8] |= code << (4 * (i % 8));
  }
  return make_uint2(w[0], w[1]);
}
// Four E4M3 codes (round to nearest even, saturating), as e4m3_code gives them.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  if (a != a || b != b || c != c || d != d)  // the conversion has another code for NaN
    return e4m3_code(a) | (e4m3_code(b) << 8) | (e4m3_code(c) << 16) | (e4m3_code(d) << 24);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (static_cast<uint32_t>(hi) << 16);
}
// Exponent and scale code of an MXFP8 block with this largest magnitude.
__device__ __forceinline__ void mxfp8_scale(float amax, float *inv, uint32_t *sc) {
  if (amax == 0.0f) {
    *inv = 0.0f;
    *sc = 0;
    return;
  }
  const int e = max(-127, min(127, floor_log2f(amax) - 8));
  *inv = pow2f(-e);
  *sc = static_cast<uint32_t>(e + 127);
}

template <bool kBf16>
struct TokenRow {
  float x[16];  // latent dims 16 l ..
  float2 r;     // RoPE dims 2 l, 2 l + 1
  float4 k;     // key dims 4 l ..
};
__device__ __forceinline__ float2 bf2(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }
template <bool kBf16>
__device__ __forceinline__ void load_token(const RaggedAppend &a, int64_t r, int lane, TokenRow<kBf16> &t) {
  if (kBf16) {
    const __nv_bfloat16 *kv = static_cast<const __nv_bfloat16 *>(a.kv) + r * a.kv_stride;
    const __nv_bfloat16 *ik = static_cast<const __nv_bfloat16 *>(a.ik) + r * a.key_stride;
    uint4 v[2];
    v[0] = __ldg(reinterpret_cast<const uint4 *>(kv + 16 * lane));
    v[1] = __ldg(reinterpret_cast<const uint4 *>(kv + 16 * lane + 8));
    const uint32_t rr = __ldg(reinterpret_cast<const uint32_t *>(kv + kLat + 2 * lane));
    const uint2 kk = __ldg(reinterpret_cast<const uint2 *>(ik + 4 * lane));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = bf2(u[j]);
        t.x[8 * i + 2 * j] = f.x;
        t.x[8 * i + 2 * j + 1] = f.y;
      }
    }
    t.r = bf2(rr);
    const float2 k0 = bf2(kk.x), k1 = bf2(kk.y);
    t.k = make_float4(k0.x, k0.y, k1.x, k1.y);
  } else {
    const float *kv = static_cast<const float *>(a.kv) + r * a.kv_stride;
    const float *ik = static_cast<const float *>(a.ik) + r * a.key_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(kv + 16 * lane + 4 * i));
      t.x[4 * i] = v.x, t.x[4 * i + 1] = v.y, t.x[4 * i + 2] = v.z, t.x[4 * i + 3] = v.w;
    }
    t.r = __ldg(reinterpret_cast<const float2 *>(kv + kLat + 2 * lane));
    t.k = __ldg(reinterpret_cast<const float4 *>(ik + 4 * lane));
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&t);
}
__device__ __forceinline__ float max_over(float v, int lanes) {  // over groups of `lanes` lanes
  for (int o = 1; o < lanes; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Where a token goes.
struct TokenPlace {
  int64_t pe;   // physical entry; -1: nothing is stored (an error, or a row of no sequence)
  int64_t pt;   // its indexer tile
  int64_t win;  // row of wcodes / wscales; -1: none
  int64_t t;
};

// Eight tokens per block.  Blocks behind the tokens' copy the older window rows, or
// (single) check the list.
template <bool kBf16>
__global__ void __launch_bounds__(256, 4) k_ragged_append_r1(RaggedAppend a, int single, int token_blocks) {
  if (static_cast<int>(blockIdx.x) >= token_blocks) {
    if (single) check_list(a, blockIdx.x - token_blocks);
    else copy_older(a, blockIdx.x - token_blocks);
    return;
  }
  const csa2_cache &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the row does not depend on its place: it is requested at once
  TokenRow<kBf16> cur;
  const int r = blockIdx.x * 8 + warp;
  if (r >= a.total) return;
  load_token(a, r, lane, cur);
  TokenPlace pl{-1, -1, -1, 0};  // (the same in every lane)
  const RaggedRow rr = ragged_row(a.cu, c.batch, a.total, a.max_new, r);
  const int b = rr.b, first = rr.first, n = rr.n;
  if (b < 0) return;
  if (n == 0) {
    if (lane == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
    return;
  }
  const int64_t t0 = c.n_tokens[b];
  const int j = r - first;
  if (!append_ok(c, t0, n, a.rope_len)) {
    if (j == 0 && lane == 0) append_fail(c, t0, n, a.rope_len, a.err);
    return;
  }
  pl.t = t0 + j;
  pl.pe = entry_at(c, b, static_cast<int>(pl.t));
  // a page holds whole indexer tiles; a dense sequence's are padded
  pl.pt = c.block_table != nullptr ? pl.pe / kIdxTile : b * idx_tiles(c.capacity) + pl.t / kIdxTile;
  if (a.win_codes != nullptr) pl.win = static_cast<int64_t>(r) + static_cast<int64_t>(kWin) * (b + 1);
  else if (j >= n - kWin) pl.win = static_cast<int64_t>(b) * kWin + (pl.t & (kWin - 1));
  __syncwarp();  // every lane has read n_tokens
  if (lane == 0) {
    if (pl.pe < 0) raise_err(a.err, CSA2_DEVERR_INDEX);
    if (single) c.n_tokens[b] = t0 + n;  // (its only token: no other warp reads it)
  }
  const bool fp8 = c.entry_format == CSA2_ENTRY_FP8, mx = c.swa_dtype == CSA2_SWA_MXFP8;
  if (pl.pe < 0 && pl.win < 0) return;
  const float2 cs = __ldg(reinterpret_cast<const float2 *>(a.rope_cs + pl.t * 64 + 2 * lane));
  rope_pair(cur.r.x, cur.r.y, cs.x, cs.y);
  // E4M3 latents, shared by a V4 entry and an MXFP8 window row
  uint4 lat8 = make_uint4(0, 0, 0, 0);
  uint32_t lat8_sc = 0;
  if ((fp8 && pl.pe >= 0) || (mx && pl.win >= 0)) {
    float amax = fabsf(cur.x[0]), inv;
#pragma unroll
    for (int j = 1; j < 16; ++j) amax = fmaxf(amax, fabsf(cur.x[j]));
    amax = max_over(amax, 2);
    mxfp8_scale(amax, &inv, &lat8_sc);
    if (amax != 0.0f) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = e4m3x4(__fmul_rn(cur.x[4 * j], inv), __fmul_rn(cur.x[4 * j + 1], inv), __fmul_rn(cur.x[4 * j + 2], inv),
                      __fmul_rn(cur.x[4 * j + 3], inv));
      lat8 = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (pl.pe >= 0) {
    if (fp8) {
      *reinterpret_cast<uint4 *>(c.lat_codes + pl.pe * 512 + 16 * lane) = lat8;
      if ((lane & 1) == 0) c.lat_scales[pl.pe * 16 + (lane >> 1)] = static_cast<uint8_t>(lat8_sc);
      reinterpret_cast<uint32_t *>(c.rope_codes + pl.pe * 128)[lane] = bf16_pair(cur.r.x, cur.r.y);
    } else {
      uint32_t sc;
      const uint2 w = nvfp4_16(cur.x, &sc);
      *reinterpret_cast<uint2 *>(c.lat_codes + pl.pe * 256 + 8 * lane) = w;
      c.lat_scales[pl.pe * 32 + lane] = static_cast<uint8_t>(sc);
      const uint32_t byte = nvfp4_pair(cur.r.x, cur.r.y, &sc);
      c.rope_codes[pl.pe * 32 + lane] = static_cast<uint8_t>(byte);
      if ((lane & 7) == 0) c.rope_scales[pl.pe * 4 + (lane >> 3)] = static_cast<uint8_t>(sc);
    }
    // the indexer key, MXFP4: block lane / 8
    const float x[4] = {cur.k.x, cur.k.y, cur.k.z, cur.k.w};
    const float amax = max_over(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))), 8);
    uint32_t codes = 0, sc = 0;
    if (amax != 0.0f) {
      const int e = max(-127, min(127, floor_log2f(amax) - 2));
      const float inv = pow2f(-e);
#pragma unroll
      for (int j = 0; j < 4; ++j) codes |= e2m1_code(__fmul_rn(x[j], inv)) << (4 * j);
      sc = static_cast<uint32_t>(e + 127);
    }
    const int m = static_cast<int>(pl.t % kIdxTile), blk = lane >> 3;
    *reinterpret_cast<uint16_t *>(c.idx_codes + idx_code_at(pl.pt, m, blk) + 2 * (lane & 7)) = static_cast<uint16_t>(codes);
    if ((lane & 7) == 0) c.idx_scales[idx_scale_at(pl.pt, m) + blk] = static_cast<uint8_t>(sc);
  }
  if (pl.win >= 0) {
    uint8_t *wc = (a.win_codes != nullptr ? a.win_codes : c.swa_codes) + pl.win * (mx ? 576 : 1152);
    if (mx) {
      uint8_t *ws = (a.win_codes != nullptr ? a.win_scales : c.swa_scales) + pl.win * kSwaScaleStride;
      *reinterpret_cast<uint4 *>(wc + 16 * lane) = lat8;
      if ((lane & 1) == 0) ws[lane >> 1] = static_cast<uint8_t>(lat8_sc);
      const float amax = max_over(fmaxf(fabsf(cur.r.x), fabsf(cur.r.y)), 16);
      float inv;
      uint32_t sc, code = 0;
      mxfp8_scale(amax, &inv, &sc);
      if (amax != 0.0f) code = e4m3x4(__fmul_rn(cur.r.x, inv), __fmul_rn(cur.r.y, inv), 0.0f, 0.0f) & 0xFFFFu;
      reinterpret_cast<uint16_t *>(wc + kLat)[lane] = static_cast<uint16_t>(code);
      if ((lane & 15) == 0) ws[16 + (lane >> 4)] = static_cast<uint8_t>(sc);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = bf16_pair(cur.x[2 * j], cur.x[2 * j + 1]);
      uint4 *d = reinterpret_cast<uint4 *>(wc + 32 * lane);
      d[0] = make_uint4(w[0], w[1], w[2], w[3]);
      d[1] = make_uint4(w[4], w[5], w[6], w[7]);
      reinterpret_cast<uint32_t *>(wc + 2 * kLat)[lane] = bf16_pair(cur.r.x, cur.r.y);
    }
  }
}

// ---------------------------------------------------------------- ratio 2: a block per token
// The compression (704 channels, fp64 softmax over four rows) is csa2_kv_append's,
// and its arithmetic is what bounds it: 32,768 tokens take 2.7 ms (csa2_kv_append
// 2.8), 370 MB at 2 % of the HBM rate with the fp64 pipe at 89 %.  Every second token
// brings an entry; the others' blocks cost next to nothing beside it.  Groups
// of NaN alone become zeros, as csa2_kv_append's encoders for ratio 2 make them.
// Blocks 0 .. total-1: one token each (its window row and, when it completes a
// pair, the entry).  single: max_new is 1 and there are no window rows to leave,
// so a token's block also finishes its sequence.
__global__ void __launch_bounds__(kEncThreads) k_ragged_append_r2(RaggedAppend a, int single) {
  const csa2_cache &c = a.c;
  if (static_cast<int>(blockIdx.x) >= a.total) {
    if (single) check_list(a, blockIdx.x - a.total);
    else copy_older(a, blockIdx.x - a.total);
    return;
  }
  __shared__ __align__(16) float row[kDcmp];
  __shared__ __align__(16) float rot[kRope];
  const int r = blockIdx.x;
  const RaggedRow rr = ragged_row(a.cu, c.batch, a.total, a.max_new, r);
  const int b = rr.b, first = rr.first, n = rr.n;
  if (b < 0) return;
  if (n == 0) {
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
  for (int i = threadIdx.x; i < kDqk; i += blockDim.x) row[i] = a.cmp.ca[static_cast<size_t>(r) * kDcmp + i];
  if (threadIdx.x < 64) rot[threadIdx.x] = a.rope_cs[t * 64 + threadIdx.x];
  __syncthreads();
  block_rope_inplace(row, rot);
  __syncthreads();
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
  if (wc != nullptr) block_encode_swa<true>(wc, ws, c.swa_dtype, row, rot);
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
    block_encode_entry<true>(c, b, e, row, rot, a.err);
  }
  // a single token's slot (t % 4) is none of those its entry was made from
  if (single) {
    store_cmp_rows(a, b, r, t);
    __syncthreads();  // every thread has read n_tokens
    if (threadIdx.x == 0) c.n_tokens[b] = t0 + n;
  }
}

// Once every token is encoded (3 us, a launch of its own: no block of the append
// knows when the last one has read the ring): the ring (from the window rows, when they were
// asked for), the compression buffer, n_tokens.  One block per sequence.
__global__ void __launch_bounds__(256) k_ragged_finish(RaggedAppend a) {
  const csa2_cache &c = a.c;
  const int b = blockIdx.x;
  int first, n;
  if (!ragged_rows(a.cu, b, a.total, a.max_new, first, n)) {
    if (threadIdx.x == 0) raise_err(a.err, CSA2_DEVERR_INDEX);
    return;
  }
  if (n == 0) return;
  const int64_t t0 = c.n_tokens[b];
  if (!block_ragged_own(a.cu, c.batch, b, first, n) || !append_ok(c, t0, n, a.rope_len)) return;
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
  int32_t *err;
};

// 8 warps, kRow rows each, in units of 8 values: lane l has latent units l and
// l + 32, lanes 0-7 the RoPE units, lanes 8-23 the key's; every store instruction
// of the latent writes a contiguous 512 B (bf16).  One thread per row first finds
// where it lies (a chain of dependent loads) for the whole block (by warps, without
// the barrier, took as long); then a warp requests all its rows before it converts
// the first.  229,000 FP4 rows to bf16 take 67 us: 412 MB, 6.1 TB/s, 90 % of the
// measured copy rate; 30,011 V4 rows to fp32 18 to 20 us (part of what they write is
// still in L2 then); 16,384 FP4 rows at listed positions 11 us (round trips).
struct RowPlace {
  int64_t pe, pt;  // physical entry and indexer tile; pe -1: zeros, -2: no row
  int32_t m;       // place in the indexer tile
};
struct RawRow {
  uint2 c[2];       // latent units l, l + 32
  uint4 x;          // lanes 0-7: RoPE, 8-23: key
  uint32_t s[2], t; // their scales
};
// Eight fp32 values: one 32 B store where the address allows it (rows of an output
// that starts on 16 B alone take two).
__device__ __forceinline__ void store_f32x8(uint8_t *dst, const float *v) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
// A unit from memory as half pairs and a scale to fp32, times the scale (exact),
// to the output row.
template <bool kBf16>
__device__ __forceinline__ void store_unit(uint8_t *dst, const uint32_t *h, float s) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
  if (kBf16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    store_f32x8(dst, v);
  }
}
__device__ __forceinline__ float e4m3_scale(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  return __low2float(*reinterpret_cast<const __half2 *>(&h));
}
template <bool kBf16, int kRow>
__global__ void __launch_bounds__(256, 4) k_kv_read(ReadArgs a) {
  __shared__ RowPlace place[8 * kRow];
  const csa2_cache &c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 8 * kRow;
  if (tid < 8 * kRow) {
    RowPlace pl{-2, 0, 0};
    const int64_t r = r0 + tid;
    // (requested before the search for the sequence, which does not need it)
    const int32_t listed = a.pos != nullptr && r < a.total ? __ldg(a.pos + r) : 0;
    RaggedRow rr{-1, 0, 0};
    if (r < a.total) rr = ragged_row(a.cu, c.batch, a.total, a.total, static_cast<int>(r));
    const int b = rr.b;
    if (b >= 0 && rr.n == 0) {
      raise_err(a.err, CSA2_DEVERR_INDEX);  // (no row: left as it was)
    } else if (b >= 0) {
      pl.pe = -1;
      const int64_t e = a.pos ? static_cast<int64_t>(listed) : a.start[b] + (r - rr.first);
      bool bad = e < 0 && a.pos == nullptr;  // a negative start
      if (e >= 0) {
        bad = e >= c.n_tokens[b] >> (c.ratio - 1) || e >= c.capacity;
        if (!bad) {
          pl.pe = entry_at(c, b, static_cast<int>(e));
          pl.m = static_cast<int>(e % kIdxTile);
          // a page holds whole indexer tiles; a dense sequence's are padded
          pl.pt = c.block_table != nullptr ? pl.pe / kIdxTile : b * idx_tiles(c.capacity) + e / kIdxTile;
          bad = pl.pe < 0;
        }
      }
      if (bad) {
        raise_err(a.err, CSA2_DEVERR_INDEX);
        pl.pe = -1;
      }
    }
    place[tid] = pl;
  }
  // sequences that have no row in the arrays (the threads without a row first)
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 256 + (255 - tid); b < c.batch; b += static_cast<int64_t>(gridDim.x) * 256) {
    int first, n;
    if (!ragged_rows(a.cu, static_cast<int>(b), a.total, a.total, first, n)) raise_err(a.err, CSA2_DEVERR_INDEX);
  }
  __syncthreads();
  const bool fp8 = c.entry_format == CSA2_ENTRY_FP8;
  const bool main = a.main != nullptr, key = a.key != nullptr;
  // lanes 0-7 have a RoPE unit, lanes 8-23 a key unit
  const bool rope = main && lane < 8, has_key = key && lane >= 8 && lane < 24;
  const int ku = lane - 8;
  constexpr int kBatch = kRow < 4 ? kRow : 4, kElt = kBf16 ? 2 : 4;  // rows in flight; bytes of a value
#pragma unroll 1
  for (int i0 = 0; i0 < kRow; i0 += kBatch) {
    RawRow raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const RowPlace &pl = place[warp * kRow + i0 + i];
      const int64_t pe = pl.pe;
      RawRow &w = raw[i];
      if (pe < 0) continue;
      if (main) {
        if (fp8) {
          const uint2 *lc = reinterpret_cast<const uint2 *>(c.lat_codes + pe * 512) + lane;
          const uint8_t *ls = c.lat_scales + pe * 16 + (lane >> 2);
          w.c[0] = __ldg(lc);
          w.c[1] = __ldg(lc + 32);
          w.s[0] = __ldg(ls);
          w.s[1] = __ldg(ls + 8);
        } else {
          const uint32_t *lc = reinterpret_cast<const uint32_t *>(c.lat_codes + pe * 256) + lane;
          const uint8_t *ls = c.lat_scales + pe * 32 + (lane >> 1);
          w.c[0].x = __ldg(lc);
          w.c[1].x = __ldg(lc + 32);
          w.s[0] = __ldg(ls);
          w.s[1] = __ldg(ls + 16);
        }
      }
      if (rope && fp8) {
        w.x = __ldg(reinterpret_cast<const uint4 *>(c.rope_codes + pe * 128) + lane);
      } else if (rope || has_key) {
        const uint8_t *src = rope ? c.rope_codes + pe * 32 + 4 * lane
                                  : c.idx_codes + idx_code_at(pl.pt, pl.m, ku >> 2) + 4 * (ku & 3);
        const uint8_t *sc = rope ? c.rope_scales + pe * 4 + (lane >> 1) : c.idx_scales + idx_scale_at(pl.pt, pl.m) + (ku >> 2);
        w.x.x = __ldg(reinterpret_cast<const uint32_t *>(src));
        w.t = __ldg(sc);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = warp * kRow + i0 + i;
      const int64_t pe = place[at].pe, r = r0 + at;
      if (pe == -2) continue;
      RawRow &w = raw[i];
      if (pe < 0) {
        w = RawRow{};  // an empty row: codes of zero, and a scale of zero (1 for E8M0: 0 x 2^-127)
        w.t = 0;
      }
      uint8_t *om = static_cast<uint8_t *>(a.main) + r * a.main_stride * kElt + 8 * kElt * lane;
      uint32_t h[4];
      if (main) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (fp8) e4m3x8_h2(w.c[k].x, w.c[k].y, h);
          else e2m1x8_h2(w.c[k].x, h);
          store_unit<kBf16>(om + 256 * kElt * k, h, fp8 ? e8m0_value(w.s[k]) : e4m3_scale(w.s[k]));
        }
      }
      if (rope && fp8) {
        if (kBf16) {
          *reinterpret_cast<uint4 *>(om + kLat * kElt) = w.x;
        } else {
          float v[8];
          bf16x8(w.x, v);
          store_f32x8(om + kLat * kElt, v);
        }
      } else if (rope || has_key) {
        uint8_t *dst = rope ? om + kLat * kElt : static_cast<uint8_t *>(a.key) + r * a.key_stride * kElt + 8 * kElt * ku;
        e2m1x8_h2(w.x.x, h);
        store_unit<kBf16>(dst, h, rope ? e4m3_scale(w.t) : e8m0_value(w.t));
      }
    }
  }
}

// One thread per 8 values of a window token: 32 windows 5 us, a launch and a round
// trip or two.
__global__ void __launch_bounds__(256) k_window_read(csa2_cache c, void *out, int bf16) {
  const uint32_t id = blockIdx.x * 256 + threadIdx.x;  // (65,535 sequences at most: below 2^30)
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
  // blocks behind the tokens'
  const int more = single ? (cache->batch + 255) / 256 : win_codes != nullptr ? csa2::kCopyBlocks * cache->batch : 0;
  static_assert(csa2::kEncThreads == 256, "the list's blocks");
  if (cache->ratio == 2) {
    csa2::k_ragged_append_r2<<<total + more, csa2::kEncThreads, 0, s>>>(a, single);
  } else {
    const int blocks = (total + 7) / 8;
    auto kern = in_dtype == CSA2_IN_BF16 ? csa2::k_ragged_append_r1<true> : csa2::k_ragged_append_r1<false>;
    kern<<<blocks + more, 256, 0, s>>>(a, single, blocks);
  }
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
  csa2::ReadArgs a{*cache, cu_rows, total, pos, start, out_main, out_key, main_stride, key_stride, err_word};
  // four rows per warp (one address phase for them, their loads in flight together)
  // once that still leaves every SM two blocks: 131,072 rows to bf16 take 43 us
  // against 47 with one; up to 32,768 both take the same (18 us), and below
  // the rule one row per warp is ahead (2,048 rows to fp32: 8.2 us against 10.2)
  const int per = total >= 64 * csa2::device_sm_count() ? 32 : 8;
  const bool bf16 = out_dtype == CSA2_OUT_BF16;
  auto kern = bf16 ? (per == 32 ? csa2::k_kv_read<true, 4> : csa2::k_kv_read<true, 1>)
                   : (per == 32 ? csa2::k_kv_read<false, 4> : csa2::k_kv_read<false, 1>);
  kern<<<(total + per - 1) / per, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
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
