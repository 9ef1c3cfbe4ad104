// csa2_fp4.cu -- rows quantised into a 4-bit block-scaled matrix (csa2_fp4_quant) and
// read back as the values they stand for (csa2_fp4_read).
//
// NV: a row's power of two r brings its largest magnitude to 2688 = 448 x 6 at most;
// then per 16 values s = E4M3(amax / 6), codes E2M1(x / (r s)).  MX: per 32 values
// e = floor(log2 amax) - 2, codes E2M1(x 2^-e).  A row with an infinity or NaN, or one
// beyond 2688 x 2^62 in NV, has the row scale NaN: whatever is computed from it is NaN.
//
// x / s in E2M1 without a division.  A quotient rounds to a code by its place among the
// grid's midpoints T (1, 3, 5 or 7 times a power of two); s has 4 significant bits.
//   bf16 x (8 bits): x and T s are integers up to 255 and 105 times powers of two, so x / s
//   is T or differs from it by 2^-8 of it at least.  x * RN(1 / s), off by 2^-23, is
//   rounded to 12 fraction bits: T where the quotient is T, on its side of T where not;
//   then the conversion instruction decides.
//   fp32 x: |x| is compared with T s, which is exact.  (The correctly rounded quotient, by
//   which the formula decides, is T only if x = T s: the next fp32 values beside T s are
//   2^-24 of it away at least, and more than half a step of T.)
//
// Bound: HBM for large matrices, a chain of loads, reductions and stores for a few rows.
#include "csa2_fp4.cuh"

namespace csa2 {
namespace {

constexpr int kQThreads = 256;

struct F4Args {
  csa2_fp4_matrix m;
  const void *x;
  int64_t stride;
  int32_t *err;
};

// |bits| of up to 32 values, and the values, from column c0 of a row; zeros behind `cols`.
template <bool kBf16>
__device__ __forceinline__ void load32(const void *row, int c0, int cols, float *v) {
  if constexpr (kBf16) {
    const uint16_t *p = static_cast<const uint16_t *>(row) + c0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (c0 + 8 * q + 8 <= cols) {
        w = __ldg(reinterpret_cast<const uint4 *>(p) + q);
      } else {
        uint32_t t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = c0 + 8 * q + i < cols ? p[8 * q + i] : 0u;
        w = make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16);
      }
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * q + 2 * i] = __uint_as_float(u[i] << 16);
        v[8 * q + 2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
  } else {
    const float *p = static_cast<const float *>(row) + c0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float4 w = make_float4(0, 0, 0, 0);
      if (c0 + 4 * q + 4 <= cols) {
        w = __ldg(reinterpret_cast<const float4 *>(p) + q);
      } else {
        if (c0 + 4 * q < cols) w.x = p[4 * q];
        if (c0 + 4 * q + 1 < cols) w.y = p[4 * q + 1];
        if (c0 + 4 * q + 2 < cols) w.z = p[4 * q + 2];
      }
      v[4 * q] = w.x;
      v[4 * q + 1] = w.y;
      v[4 * q + 2] = w.z;
      v[4 * q + 3] = w.w;
    }
  }
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
template <int kN>
__device__ __forceinline__ uint32_t top_bits(const float *v) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) t = max(t, abs_bits(v[i]));
  return t;
}
// Eight values to eight E2M1 codes (low nibble first), RNE, saturating: the conversion
// instruction takes two values, the first argument into the high nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float *y) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// 16 values y (already divided by the row's power of two) into two words and an E4M3 scale.
template <bool kBf16>
__device__ __forceinline__ void nv16(const float *y, uint32_t *w, uint32_t *sc) {
  const float amax = __uint_as_float(top_bits<16>(y));
  const uint32_t code = e4m3_code(__fdiv_rn(amax, 6.0f));
  const float s = e4m3_value(code);
  *sc = code;
  w[0] = w[1] = 0;
  if (code == 0) return;
  if constexpr (kBf16) {
    const float inv = __frcp_rn(s);
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __uint_as_float((__float_as_uint(__fmul_rn(y[i], inv)) + 0x400u) & ~0x7FFu);
    w[0] = e2m1x8(q);
    w[1] = e2m1x8(q + 8);
  } else {
    const float t0 = 0.25f * s, t1 = 0.75f * s, t2 = 1.25f * s, t3 = 1.75f * s, t4 = 2.5f * s, t5 = 3.5f * s, t6 = 5.0f * s;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(y[i]);
      uint32_t c = (a > t0) + (a >= t1) + (a > t2) + (a >= t3) + (a > t4) + (a >= t5) + (a > t6);
      c |= (__float_as_uint(y[i]) >> 28) & 8u;
      w[i >> 3] |= c << (4 * (i & 7));
    }
  }
}

// One block: kRows consecutive rows (8, so that a piece's 16 bytes of theirs are whole
// 128 B lines; or 1, for few rows).  A thread takes 32 values of a row at a time.
template <bool kNv, bool kBf16, int kRows>
__global__ void __launch_bounds__(kQThreads) k_fp4_quant(F4Args a) {
  constexpr int kElt = kBf16 ? 2 : 4;
  __shared__ uint32_t top[8], part[8];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rows = a.m.rows, cols = a.m.cols;
  const int row0 = blockIdx.x * kRows;
  const int row = row0 + (kRows == 8 ? t & 7 : 0);  // this thread's, once it writes
  const uint8_t *x = static_cast<const uint8_t *>(a.x);
  float v[32];
  uint32_t bad = 0;
  float back = 1.0f;  // 2^-(row exponent)
  if constexpr (kNv) {
    if constexpr (kRows == 8) {  // a warp per row
      uint32_t m = 0;
      if (row0 + warp < rows) {
        const uint8_t *src = x + (row0 + warp) * a.stride * kElt;
        for (int c = 32 * lane; c < cols; c += 1024) {
          load32<kBf16>(src, c, cols, v);
          m = max(m, top_bits<32>(v));
        }
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) top[warp] = m;
    } else {
      uint32_t m = 0;
      for (int c = 32 * t; c < cols; c += 32 * kQThreads) {
        load32<kBf16>(x + row * a.stride * kElt, c, cols, v);
        m = max(m, top_bits<32>(v));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) part[warp] = m;
      __syncthreads();
      if (t < 8) {
        m = __reduce_max_sync(0xffu, part[t]);
        if (t == 0) top[0] = m;
      }
    }
    __syncthreads();
    const uint32_t m = top[kRows == 8 ? t & 7 : 0];
    // amax = f 2^E: 2688 = 1.3125 x 2^11
    int e = m ? floor_log2f(__uint_as_float(m)) : 0;
    if (m >= 0x00800000u) e += (m & 0x7FFFFFu) > 0x280000u ? -10 : -11;
    e = m ? max(e, -62) : 0;
    bad = e > 62 || m >= 0x7F800000u;
    back = bad ? 0.0f : pow2f(-e);
    if (row < rows && t < kRows) {
      a.m.row_scales[row] = bad ? __uint_as_float(0x7FC00000u) : pow2f(e);
      if (bad) raise_err(a.err, CSA2_DEVERR_NAN);
    }
  }
  const int ct = static_cast<int>(f4_col_tiles(cols)), pieces = 4 * ct;
  const int m = row % kF4Rows;
  const int64_t tile0 = static_cast<int64_t>(row / kF4Rows) * ct;
  if (row < rows) {
    for (int p = kRows == 8 ? t >> 3 : t; p < pieces; p += kQThreads / kRows) {
      load32<kBf16>(x + row * a.stride * kElt, 32 * p, cols, v);
      uint32_t w[4];
      uint8_t *rec = a.m.tiles + (tile0 + (p >> 2)) * f4_tile_bytes(kNv), *sc = rec + kF4CodeBytes + f4_scale_at(m);
      if constexpr (kNv) {
        uint32_t s0, s1;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = bad ? 0.0f : __fmul_rn(v[i], back);
        nv16<kBf16>(v, w, &s0);
        nv16<kBf16>(v + 16, w + 2, &s1);
        *reinterpret_cast<uint16_t *>(sc + 512 * ((p >> 1) & 1) + 2 * (p & 1)) = static_cast<uint16_t>(s0 | s1 << 8);
      } else {
        const uint32_t top32 = top_bits<32>(v);
        uint32_t code = 0;
        w[0] = w[1] = w[2] = w[3] = 0;
        if (top32 >= 0x7F800000u) {
          bad = 1;
        } else if (top32 != 0) {
          const int e = max(floor_log2f(__uint_as_float(top32)) - 2, -127);
          const float inv = pow2f(-e);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(v[i], inv);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = e2m1x8(v + 8 * i);
          code = static_cast<uint32_t>(e + 127);
        }
        sc[p & 3] = static_cast<uint8_t>(code);
      }
      *reinterpret_cast<uint4 *>(rec + (p & 3) * 2048 + m * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if constexpr (!kNv) {
    if (t < 8) top[t] = 0;
    __syncthreads();
    if (bad) atomicOr(&top[kRows == 8 ? t & 7 : 0], 1u);
    __syncthreads();
    if (row < rows && t < kRows) {
      a.m.row_scales[row] = top[t] ? __uint_as_float(0x7FC00000u) : 1.0f;
      if (top[t]) raise_err(a.err, CSA2_DEVERR_NAN);
    }
  }
}

// A warp: 8 rows x 32 columns at a time (128 B of codes in, 64 B per row out).
template <bool kNv, bool kBf16>
__global__ void __launch_bounds__(256) k_fp4_read(csa2_fp4_matrix mx, void *out, int64_t stride) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ct = static_cast<int>(f4_col_tiles(mx.cols)), pieces = (mx.cols + 31) / 32;
  const int row = blockIdx.x * 8 + (lane >> 2), u = lane & 3;
  if (row >= mx.rows) return;
  const int m = row % kF4Rows;
  const float r = mx.row_scales[row];
  const int64_t tile0 = static_cast<int64_t>(row / kF4Rows) * ct;
  for (int p = blockIdx.y * 8 + warp; p < pieces; p += 8 * gridDim.y) {
    const uint8_t *rec = mx.tiles + (tile0 + (p >> 2)) * f4_tile_bytes(kNv), *sc = rec + kF4CodeBytes + f4_scale_at(m);
    const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + (p & 3) * 2048 + m * 16 + 4 * u);
    const float s = kNv ? e4m3_value(sc[512 * ((p >> 1) & 1) + 2 * (p & 1) + (u >> 1)]) * r : e8m0_value(sc[p & 3]) * r;
    uint32_t h[4];
    e2m1x8_h2(w, h);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[i]));
      v[2 * i] = f.x * s;
      v[2 * i + 1] = f.y * s;
    }
    const int c = 32 * p + 8 * u;
    const int64_t at = row * stride + c;
    if (c + 8 <= mx.cols) {
      if constexpr (kBf16) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          o[i] = *reinterpret_cast<uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < mx.cols) {
          if constexpr (kBf16) static_cast<__nv_bfloat16 *>(out)[at + i] = __float2bfloat16_rn(v[i]);
          else static_cast<float *>(out)[at + i] = v[i];
        }
    }
  }
}

}  // namespace

csa2_status check_fp4(const csa2_fp4_matrix *m, const char *name) {
  CSA2_REQUIRE(m != nullptr, CSA2_ERR_NULL, "%s is NULL", name);
  CSA2_REQUIRE(m->rows >= 0 && m->rows <= (1 << 24), CSA2_ERR_SHAPE, "%s: rows %d outside 0..2^24", name, m->rows);
  CSA2_REQUIRE(m->cols >= 1 && m->cols <= (1 << 17), CSA2_ERR_SHAPE, "%s: cols %d outside 1..2^17", name, m->cols);
  CSA2_REQUIRE(m->format == CSA2_FP4_NV || m->format == CSA2_FP4_MX, CSA2_ERR_RANGE, "%s: format %d", name, m->format);
  if (m->rows == 0) return CSA2_OK;
  CSA2_REQUIRE(m->tiles && m->row_scales, CSA2_ERR_NULL, "%s: a plane is NULL", name);
  CSA2_REQUIRE(aligned16(m->tiles) && aligned16(m->row_scales), CSA2_ERR_ALIGN,
               "%s: a plane is not 16-byte aligned", name);
  return CSA2_OK;
}

}  // namespace csa2

extern "C" {

using csa2::cuda_status;

size_t csa2_fp4_plane_bytes(int32_t rows, int32_t cols, int32_t format, int32_t plane) {
  if (rows < 0 || cols <= 0 || (format != CSA2_FP4_NV && format != CSA2_FP4_MX)) return 0;
  const size_t tiles = static_cast<size_t>(csa2::f4_row_tiles(rows)) * csa2::f4_col_tiles(cols);
  switch (plane) {
    case 0: return tiles * csa2::f4_tile_bytes(format == CSA2_FP4_NV);
    case 1: return static_cast<size_t>(csa2::f4_row_tiles(rows)) * csa2::kF4Rows * sizeof(float);
  }
  return 0;
}

csa2_status csa2_fp4_quant(const csa2_fp4_matrix *m, const void *x, int64_t x_stride, int32_t in_dtype, int32_t *err_word,
                           csa2_stream_t stream) {
  csa2_status st = csa2::check_fp4(m, "m");
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(in_dtype == CSA2_IN_F32 || in_dtype == CSA2_IN_BF16, CSA2_ERR_RANGE, "in_dtype %d", in_dtype);
  CSA2_REQUIRE(x_stride >= m->cols && x_stride % 8 == 0, CSA2_ERR_SHAPE, "x_stride %lld must be a multiple of 8, %d at least",
               static_cast<long long>(x_stride), m->cols);
  if (m->rows == 0) return CSA2_OK;
  CSA2_REQUIRE_PTR(x);
  const csa2::F4Args a{*m, x, x_stride, err_word};
  const bool nv = m->format == CSA2_FP4_NV, bf = in_dtype == CSA2_IN_BF16;
  const bool many = m->rows >= 8 * csa2::device_sm_count();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define CSA2_Q(NV, BF)                                                                               \
  (many ? csa2::k_fp4_quant<NV, BF, 8><<<(m->rows + 7) / 8, csa2::kQThreads, 0, s>>>(a)              \
        : csa2::k_fp4_quant<NV, BF, 1><<<m->rows, csa2::kQThreads, 0, s>>>(a))
  if (nv) bf ? CSA2_Q(true, true) : CSA2_Q(true, false);
  else bf ? CSA2_Q(false, true) : CSA2_Q(false, false);
#undef CSA2_Q
  return cuda_status(cudaGetLastError(), "csa2_fp4_quant launch");
}

csa2_status csa2_fp4_read(const csa2_fp4_matrix *m, void *out, int64_t out_stride, int32_t out_dtype, csa2_stream_t stream) {
  csa2_status st = csa2::check_fp4(m, "m");
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(out_dtype == CSA2_OUT_F32 || out_dtype == CSA2_OUT_BF16, CSA2_ERR_RANGE, "out_dtype %d", out_dtype);
  CSA2_REQUIRE(out_stride >= m->cols && out_stride % 8 == 0, CSA2_ERR_SHAPE,
               "out_stride %lld must be a multiple of 8, %d at least", static_cast<long long>(out_stride), m->cols);
  if (m->rows == 0) return CSA2_OK;
  CSA2_REQUIRE_PTR(out);
  const int pieces = (m->cols + 31) / 32, row_blocks = (m->rows + 7) / 8;
  int split = (4 * csa2::device_sm_count() + row_blocks - 1) / row_blocks;  // few rows: their pieces over more blocks
  split = split < 1 ? 1 : split > (pieces + 7) / 8 ? (pieces + 7) / 8 : split;
  const dim3 grid(row_blocks, split);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = out_dtype == CSA2_OUT_BF16;
  if (m->format == CSA2_FP4_NV) {
    if (bf) csa2::k_fp4_read<true, true><<<grid, 256, 0, s>>>(*m, out, out_stride);
    else csa2::k_fp4_read<true, false><<<grid, 256, 0, s>>>(*m, out, out_stride);
  } else {
    if (bf) csa2::k_fp4_read<false, true><<<grid, 256, 0, s>>>(*m, out, out_stride);
    else csa2::k_fp4_read<false, false><<<grid, 256, 0, s>>>(*m, out, out_stride);
  }
  return cuda_status(cudaGetLastError(), "csa2_fp4_read launch");
}

}  // extern "C"
