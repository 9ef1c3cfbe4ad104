// csa2_fp4.cu -- rows quantised into a 4-bit block-scaled matrix (csa2_fp4_quant) and
// read back as the values they stand for (csa2_fp4_read).
//
// NV: a row's power of two r brings its largest magnitude to 2688 = 448 x 6 at most;
// then per 16 values s = E4M3(amax / 6), codes E2M1(x / (r s)).  MX: per 32 values
// e = floor(log2 amax) - 2, codes E2M1(x 2^-e).  A row with an infinity or NaN, or one
// beyond 2688 x 2^62 in NV, has the row scale NaN: whatever is computed from it is NaN.
//
// x / s in E2M1 without a division.  A quotient rounds to a code by its place among the
// grid's midpoints T (1, 3, 5 or 7 times a power of two, 1/4 at least); s has 4 significant
// bits.
//   bf16 x (8 bits): x and T s are integers up to 255 and 105 times powers of two, so x / s
//   is T or differs from it by 2^-8 of it, 2^-10, at least.  x * (1 / s), off by 2^-21 at
//   most, is rounded to a multiple of 2^-12 (by adding 1.5 x 2^11 and taking it away): T
//   where the quotient is T, on its side of T where not; then the conversion instruction
//   decides.  In the same way the scale, amax / 6 in E4M3 (midpoints of 5 bits), comes from
//   a product with 1 / 6 rounded to 12 fraction bits.
//   fp32 x: y = x (1 / s), then y + (x - y s) (1 / s), the remainder exact: off by less than
//   2^-40 of the quotient before its rounding.  If x = T s that is T.  Else the quotient is
//   2^-24 of T away from it at least (the next fp32 values beside T s), more than half a
//   step of T: the rounded one lies on the same side.  The scale comes from amax and 1 / 6 in
//   the same way (equal to the rounded quotient for every mantissa: tests/test_fp4_scale.py).
//
// Bound: HBM for large matrices, a chain of loads, reductions and stores for a few rows.
// Measured (in a graph): 12,288 x 4,096 bf16 to NV 23.2 us (5.6 TB/s), read back 22.2 us (5.8
// TB/s); 8,192 x 4,096 bf16 14.2 us (6.1 TB/s), fp32 26.5 us (5.8), to MX 14.1 and 25.9, read 12.2
// us (7.0, L2 holds a part); 32 rows 1.9 us.  At 11.6 instructions per value the first took 31 us, at 14 compares per fp32 value 42
// of 8,192 x 4,096, and with divisions 28: the conversions above are what brought them near the
// copy rate.  (Figures from one box to the next differ by 4 %.)
#include <type_traits>

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

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
template <int kN>
__device__ __forceinline__ uint32_t top_bits(const float *v) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) t = max(t, abs_bits(v[i]));
  return t;
}
// Eight values to eight E2M1 codes (low nibble first), RNE, saturating: the conversion
// instruction takes two values, the first argument into the high nibble.  Called outside
// of branches and its result chosen afterwards: with a call inside a branch the compiler
// (CUDA 13.0) gave all four conversions the same values.
__device__ __forceinline__ uint32_t e2m1x8(const float *y) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// (a, b) x inv rounded to multiples of 2^-12, with a's and b's signs: two values an instruction (one
// each, the signs took 22.4 -> 24.2 us for 12,288 x 4,096 bf16; so 22.7).
__device__ __forceinline__ void round2(float a, float b, float inv, float *q) {
  constexpr float kGrid = 1.5f * 2048.0f;  // what is added to it is rounded to a multiple of 2^-12
  uint64_t v, k, g, m;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(k) : "f"(inv));
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(g) : "f"(kGrid));
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(m) : "f"(-kGrid));
  asm("fma.rn.f32x2 %0, %0, %1, %2;\n add.rn.f32x2 %0, %0, %3;\n" : "+l"(v) : "l"(k), "l"(g), "l"(m));
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(q[0]), "=f"(q[1]) : "l"(v));
  q[0] = copysignf(q[0], a);  // (-0 plus the grid and back is +0)
  q[1] = copysignf(q[1], b);
}

// Eight values of a group with scale s of a row with power of two 2^e to eight codes (see
// the file's head), zeros if s is 0; back = 2^-e, fore = 2^e.  Both only shift exponents,
// so they go with 1 / s, or with T s, instead of with every value.  The sign is the value's
// own, as in every E2M1 code of this library: what is rounded here can leave a zero's behind.
template <bool kBf16>
__device__ __forceinline__ uint32_t nv8(const float *x, float s, float back, float fore) {
  if constexpr (kBf16) {
    float inv, q[8];
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(s));
    inv = __fmul_rn(inv, back);
#pragma unroll
    for (int i = 0; i < 8; i += 2) round2(x[i], x[i + 1], inv, q + i);
    const uint32_t w = e2m1x8(q);
    return s != 0.0f ? w : 0u;
  } else {
    float inv, q[8];
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(s));
    inv = __fmul_rn(inv, back);
    const float u = __fmul_rn(s, fore);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __fmul_rn(x[i], inv);
      q[i] = __fmaf_rn(__fmaf_rd(-y, u, x[i]), inv, y);  // (the remainder is exact; one of 0 is -0 rounded down, which leaves y's sign)
    }
    const uint32_t w = e2m1x8(q);
    return s != 0.0f ? w : 0u;
  }
}
// The scale byte of a group with largest magnitude amax, and its value.
template <bool kBf16>
__device__ __forceinline__ uint32_t nv_scale(float amax, float back, float &s) {
  const float a = __fmul_rn(amax, back);
  float y;
  if constexpr (kBf16) y = __uint_as_float((__float_as_uint(__fmul_rn(a, 1.0f / 6.0f)) + 0x400u) & ~0x7FFu);
  else y = __fmul_rn(a, 1.0f / 6.0f), y = __fmaf_rn(__fmaf_rn(-6.0f, y, a), 1.0f / 6.0f, y);
  uint16_t c;
  uint32_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(c) : "f"(0.0f), "f"(y));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(c));
  s = __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
  return c;
}
template <int kN>
__device__ __forceinline__ float top_abs(const float *v) {
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) t = fmaxf(t, fabsf(v[i]));
  return t;
}

// A row's power of two from its largest magnitude's bits: the exponent, and whether the
// row is beyond the format.
__device__ __forceinline__ int row_exponent(uint32_t m, uint32_t &bad) {
  // amax = f 2^E: 2688 = 1.3125 x 2^11
  int e = m ? floor_log2f(__uint_as_float(m)) : 0;
  if (m >= 0x00800000u) e += (m & 0x7FFFFFu) > 0x280000u ? -10 : -11;
  e = m ? max(e, -62) : 0;
  bad = e > 62 || m >= 0x7F800000u;
  return e;
}
constexpr uint32_t kNan = 0x7FC00000u;

// 32 values of a group to 16 bytes of codes and, returned, their E8M0 scale.
__device__ __forceinline__ uint32_t mx32(float *v, uint32_t &bad, uint32_t *w) {
  const uint32_t g = top_bits<32>(v);
  bad |= g >= 0x7F800000u;
  const bool some = g != 0 && g < 0x7F800000u;
  const int e = some ? max(floor_log2f(__uint_as_float(g)) - 2, -127) : 0;
  const float inv = pow2f(-e);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = some ? __fmul_rn(v[i], inv) : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e2m1x8(v + 8 * i);
  return some ? static_cast<uint32_t>(e + 127) : 0u;
}

// Eight values of a row from column c0 (bf16 or fp32; zeros behind `cols`).
template <bool kBf16>
__device__ __forceinline__ void load8(const uint8_t *row, int c0, int cols, float *v) {
  if constexpr (kBf16) {
    uint4 w = make_uint4(0, 0, 0, 0);
    const uint16_t *p = reinterpret_cast<const uint16_t *>(row) + c0;
    if (c0 + 8 <= cols) {
      w = *reinterpret_cast<const uint4 *>(p);
    } else {
      uint32_t t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = c0 + i < cols ? p[i] : 0u;
      w = make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16);
    }
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    const float *p = reinterpret_cast<const float *>(row) + c0;
    if (c0 + 8 <= cols) {
      const float4 x = reinterpret_cast<const float4 *>(p)[0], y = reinterpret_cast<const float4 *>(p)[1];
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c0 + i < cols ? p[i] : 0.0f;
    }
  }
}
// Few rows: a block per row.  A lane takes 8 values, two lanes a group of 16 (NV), four
// one of 32 (MX), so a warp's loads are one run; a row of up to kIter x 2048 values stays
// in registers between the maximum and the codes, longer ones than 4 x 2048 are read twice.
template <bool kNv, bool kBf16, int kIter>
__global__ void __launch_bounds__(kQThreads) k_fp4_quant_row(F4Args a) {
  constexpr int kHeld = kIter * 8 * kQThreads;
  constexpr int kElt = kBf16 ? 2 : 4;
  __shared__ uint32_t part[8];
  next_may_start();
  wait_for_previous();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, row = blockIdx.x, cols = a.m.cols;
  const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.stride * kElt;
  const int ct = static_cast<int>(f4_col_tiles(cols)), all = ct * kF4Cols, m = row % kF4Rows;
  uint8_t *tiles = a.m.tiles + static_cast<int64_t>(row / kF4Rows) * ct * f4_tile_bytes(kNv);
  float v[kIter][8];
  uint32_t bad = 0;
  float back = 1.0f, fore = 1.0f;  // 2^-e and 2^e, e the row's exponent
  const bool held = all <= kHeld;
  if (kNv || held) {
    uint32_t top = 0;
    for (int c0 = 0; c0 < all; c0 += kHeld) {
#pragma unroll
      for (int i = 0; i < kIter; ++i) load8<kBf16>(x, c0 + 8 * (t + kQThreads * i), cols, v[i]);
#pragma unroll
      for (int i = 0; i < kIter; ++i) top = max(top, top_bits<8>(v[i]));
    }
    if constexpr (kNv) {
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) part[warp] = top;
      __syncthreads();
      top = part[lane & 7];
      top = __reduce_max_sync(0xffffffffu, top);
      const int e = row_exponent(top, bad);
      back = pow2f(bad ? 0 : -e);
      fore = pow2f(bad ? 0 : e);
      if (t == 0) {
        a.m.row_scales[row] = bad ? __uint_as_float(kNan) : pow2f(e);
        if (bad) raise_err(a.err, CSA2_DEVERR_NAN);
      }
    }
  }
  for (int c0 = 0; c0 < all; c0 += kHeld) {
    if (!held) {
#pragma unroll
      for (int i = 0; i < kIter; ++i) load8<kBf16>(x, c0 + 8 * (t + kQThreads * i), cols, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int c = c0 + 8 * (t + kQThreads * i);  // (tiles are whole groups of 16 lanes)
      uint32_t code = 0, w = 0;
      if constexpr (kNv) {
        float g = top_abs<8>(v[i]);
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
        float sv;
        code = nv_scale<kBf16>(g, back, sv);
        w = nv8<kBf16>(v[i], sv, back, fore);
      } else {
        uint32_t g = top_bits<8>(v[i]);
        g = max(g, __shfl_xor_sync(0xffffffffu, g, 1));
        g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
        bad |= g >= 0x7F800000u;
        const bool some = g != 0 && g < 0x7F800000u;
        const int e = some ? max(floor_log2f(__uint_as_float(g)) - 2, -127) : 0;
        const float inv = pow2f(-e);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = some ? __fmul_rn(v[i][j], inv) : 0.0f;
        w = e2m1x8(y);
        code = some ? static_cast<uint32_t>(e + 127) : 0u;
      }
      if (c < all) {
        const int p = c / 32;  // the piece; its scales
        uint8_t *rec = tiles + static_cast<int64_t>(p >> 2) * f4_tile_bytes(kNv), *sc = rec + kF4CodeBytes + f4_scale_at(m);
        if constexpr (kNv) {
          if ((lane & 1) == 0) sc[512 * ((p >> 1) & 1) + 2 * (p & 1) + ((lane >> 1) & 1)] = static_cast<uint8_t>(code);
        } else {
          if ((lane & 3) == 0) sc[p & 3] = static_cast<uint8_t>(code);
        }
        *reinterpret_cast<uint32_t *>(rec + (p & 3) * 2048 + m * 16 + 4 * (lane & 3)) = w;
      }
    }
  }
  if constexpr (!kNv) {
    bad = __syncthreads_or(bad);
    if (t == 0) {
      a.m.row_scales[row] = bad ? __uint_as_float(kNan) : 1.0f;
      if (bad) raise_err(a.err, CSA2_DEVERR_NAN);
    }
  }
}

// Largest magnitude's bits (or a NaN's) of the values in a word: two bf16 or one fp32.
template <bool kBf16>
__device__ __forceinline__ uint32_t word_top(uint32_t m, uint32_t w) {
  if constexpr (kBf16) {  // m: two maxima, of any sign
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(m), "r"(w));
    return r;
  } else {
    return max(m, w & 0x7FFFFFFFu);
  }
}

// Two or one pieces of 32 values to their records: codes and scales of row m of a tile.
// A thread takes the four groups of 8 values of a piece in the order k ^ turn, which lets
// lanes whose pieces lie in the same banks read different ones (kTurns: which of turn's
// bits may be set).
template <bool kNv, bool kBf16, int kG, int kTurns>
__device__ __forceinline__ void put_pieces(uint8_t *tiles, const uint8_t *src, int p, int have, int m, float back, float fore, int turn, uint32_t &bad) {
  uint8_t *rec = tiles + static_cast<int64_t>(p >> 2) * f4_tile_bytes(kNv), *sc = rec + kF4CodeBytes + f4_scale_at(m);
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < kG; ++i) {
    uint32_t w[4], c[2];
    if constexpr (kNv) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float v[16], s;
        load8<kBf16>(src, 32 * (p + i) + 8 * (2 * g ^ turn), have, v);
        load8<kBf16>(src, 32 * (p + i) + 8 * (2 * g + 1 ^ turn), have, v + 8);
        c[g] = nv_scale<kBf16>(top_abs<16>(v), back, s);
        w[2 * g] = nv8<kBf16>(v, s, back, fore);
        w[2 * g + 1] = nv8<kBf16>(v + 8, s, back, fore);
      }
    } else {
      float v[32];
#pragma unroll
      for (int k = 0; k < 4; ++k) load8<kBf16>(src, 32 * (p + i) + 8 * (k ^ turn), have, v + 8 * k);
      c[0] = mx32(v, bad, w);
    }
    if constexpr (kTurns & 1) {
      const uint32_t a = w[0], b = w[2];
      w[0] = turn & 1 ? w[1] : w[0], w[1] = turn & 1 ? a : w[1];
      w[2] = turn & 1 ? w[3] : w[2], w[3] = turn & 1 ? b : w[3];
    }
    if constexpr (kTurns & 2) {
      const uint32_t a = w[0], b = w[1], d = c[0];
      w[0] = turn & 2 ? w[2] : w[0], w[2] = turn & 2 ? a : w[2];
      w[1] = turn & 2 ? w[3] : w[1], w[3] = turn & 2 ? b : w[3];
      if constexpr (kNv) c[0] = turn & 2 ? c[1] : c[0], c[1] = turn & 2 ? d : c[1];
    }
    if constexpr (kNv) code |= (c[0] | c[1] << 8) << (16 * i);
    else code |= c[0] << (8 * i);
    *reinterpret_cast<uint4 *>(rec + ((p + i) & 3) * 2048 + m * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  sc += kNv ? 512 * ((p >> 1) & 1) + 2 * (p & 1) : p & 3;
  if constexpr (kNv && kG == 2) *reinterpret_cast<uint32_t *>(sc) = code;
  else if constexpr (kNv || kG == 2) *reinterpret_cast<uint16_t *>(sc) = static_cast<uint16_t>(code);
  else *sc = static_cast<uint8_t>(code);
}

// Many short rows to NV, and rows too long for shared memory: a block per 8 rows, whose
// 16 bytes of a piece are a whole 128 B line.  kStaged: the rows are read once, coalesced,
// a warp per row, into shared memory (row pitch an odd number of 16 bytes, so that 8 rows'
// loads meet no bank twice); else a second time (NV) through the caches.
template <bool kNv, bool kBf16, bool kStaged>
__global__ void __launch_bounds__(kQThreads, kNv ? 4 : 3) k_fp4_quant_rows(F4Args a, int pitch) {
  constexpr int kElt = kBf16 ? 2 : 4, kRows = 8;
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ uint32_t top[kRows];
  next_may_start();
  wait_for_previous();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, rows = a.m.rows, cols = a.m.cols;
  const int row0 = blockIdx.x * kRows, r8 = t % kRows, row = row0 + r8;  // row: this thread's, once it writes
  const uint8_t *x = static_cast<const uint8_t *>(a.x);
  const int ct = static_cast<int>(f4_col_tiles(cols)), pieces = 4 * ct, m = row % kF4Rows;
  uint32_t bad = 0;
  float back = 1.0f, fore = 1.0f;  // 2^-e and 2^e, e the row's exponent
  if constexpr (kNv) {
    uint32_t big = 0;
    if (row0 + warp < rows) {
      const uint8_t *src = x + (row0 + warp) * a.stride * kElt;
      const int whole = cols * kElt & ~15;
#pragma unroll 8
      for (int c = 16 * lane; c < whole; c += 512) {
        const uint4 u = load_now(reinterpret_cast<const uint4 *>(src + c));
        if constexpr (kStaged) *reinterpret_cast<uint4 *>(stage + warp * pitch + c) = u;
        big = word_top<kBf16>(word_top<kBf16>(word_top<kBf16>(word_top<kBf16>(big, u.x), u.y), u.z), u.w);
      }
      // the last values, and zeros to the end of the last tile
      for (int c = whole / kElt + lane; c < 32 * pieces; c += 32) {
        const uint32_t u = c >= cols ? 0u : kBf16 ? reinterpret_cast<const uint16_t *>(src)[c] : reinterpret_cast<const uint32_t *>(src)[c];
        big = word_top<kBf16>(big, u);
        if constexpr (kStaged) {
          if constexpr (kBf16) reinterpret_cast<uint16_t *>(stage + warp * pitch)[c] = static_cast<uint16_t>(u);
          else reinterpret_cast<uint32_t *>(stage + warp * pitch)[c] = u;
        }
      }
    }
    if constexpr (kBf16) big = max(big << 16 & 0x7FFF0000u, big & 0x7FFF0000u);
    big = __reduce_max_sync(0xffffffffu, big);
    if (lane == 0) top[warp] = big;
    __syncthreads();
    const int e = row_exponent(top[r8], bad);
    back = pow2f(bad ? 0 : -e), fore = pow2f(bad ? 0 : e);
  }
  uint8_t *tiles = a.m.tiles + static_cast<int64_t>(row / kF4Rows) * ct * f4_tile_bytes(kNv);
  const uint8_t *src = kStaged ? stage + r8 * pitch : x + row * a.stride * kElt;
  for (int p = 2 * (t / kRows); p < pieces && row < rows; p += 2 * (kQThreads / kRows))
    put_pieces<kNv, kBf16, 2, 0>(tiles, src, p, kStaged ? 32 * pieces : cols, m, back, fore, 0, bad);
  if constexpr (!kNv) {
    if (t < kRows) top[t] = 0;
    __syncthreads();
    if (bad) atomicOr(&top[r8], 1u);
    __syncthreads();
    bad = top[r8];
  }
  if (row < rows && t < kRows) {
    a.m.row_scales[row] = bad ? __uint_as_float(kNan) : fore;
    if (bad) raise_err(a.err, CSA2_DEVERR_NAN);
  }
}

// The others: persistent blocks, kRows rows at a time, which come by bulk copies into one of
// two buffers while the other one's are quantised.  8,000 rows of 7,224 bf16 to NV 28.9 us (one
// buffer filled by loads, a block per 4 rows 44); fp32 of 4,104 26.3 (45.6; with the banks met
// up to four times and divisions 33).  A thread takes one piece of 32 values a step (so that
// the last, partial step is short), two of fp32 rows to MX, whose steps are short anyway.
struct RowsSync {
  uint64_t full[2];
  uint32_t part[kQThreads / 32];
};
template <bool kNv, bool kBf16, int kRows>
__global__ void __launch_bounds__(kQThreads, 3) k_fp4_quant_piped(F4Args a, int pitch) {
  constexpr int kElt = kBf16 ? 2 : 4, kPolls = 200;  // suspended polls of <= 1 ms each
  constexpr int kG = kNv || kBf16 ? 1 : 2, kParts = 8 / kRows;
  using Word = std::conditional_t<kBf16, uint16_t, uint32_t>;
  // Eight lanes that read 16 bytes at once are of kRows rows, 16 bytes (times an odd number)
  // apart in the banks, and of 8 / kRows pieces, 64 bytes (bf16) or 0 apart.  (8 pieces of an
  // fp32 row still meet twice.)
  constexpr int kTurns = kRows == 8 ? 0 : kRows == 4 ? (kBf16 ? 0 : 2) : kRows == 2 && kBf16 ? 2 : 3;
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ __align__(8) RowsSync sy;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rows = a.m.rows, cols = a.m.cols, ct = static_cast<int>(f4_col_tiles(cols)), pieces = 4 * ct;
  const int whole = cols * kElt & ~15, w0 = whole / kElt, tail = cols - w0;  // what the copies bring; the values behind it, < 8
  const int items = (rows + kRows - 1) / kRows, per = static_cast<int>(gridDim.x), r8 = t % kRows;
  const uint8_t *x = static_cast<const uint8_t *>(a.x);
  if (t == 0) {
    tc::mbar_init(&sy.full[0], 1);
    tc::mbar_init(&sy.full[1], 1);
    tc::fence_mbar_init();
  }
  for (int i = 0; i < 2 * kRows; ++i)  // zeros to the end of the last tile, once
    for (int c = cols + t; c < 32 * pieces; c += kQThreads) reinterpret_cast<Word *>(stage + i * pitch)[c] = 0;
  __syncthreads();
  next_may_start();
  wait_for_previous();
  auto fetch = [&](int item, int b) {
    const int n = min(kRows, rows - item * kRows);
    tc::mbar_expect_tx(&sy.full[b], n * whole);
    for (int i = 0; i < n && whole > 0; ++i)
      tc::bulk_load(tc::smem_addr(stage + (b * kRows + i) * pitch), x + (item * kRows + i) * a.stride * kElt, whole, &sy.full[b]);
  };
  // the last values of a row, taken an item ahead: thread (row, value) of the first 8 kRows
  const int tr = t / 8, tc8 = t % 8;
  auto last = [&](int item) -> Word {
    const int row = item * kRows + tr;
    return tr < kRows && tc8 < tail && row < rows ? reinterpret_cast<const Word *>(x + row * a.stride * kElt)[w0 + tc8] : 0;
  };
  Word end = last(blockIdx.x);
  if (t == 0)
    for (int b = 0; b < 2; ++b)
      if (static_cast<int>(blockIdx.x) + b * per < items) fetch(blockIdx.x + b * per, b);
  int it = 0;
  for (int item = blockIdx.x; item < items; item += per, ++it) {
    const int row = item * kRows + r8, buf = it & 1, m = row % kF4Rows;
    uint8_t *st = stage + buf * kRows * pitch;
    if (tr < kRows && tc8 < tail) reinterpret_cast<Word *>(st + tr * pitch)[w0 + tc8] = end;
    const bool ok = tc::mbar_wait_bounded(&sy.full[buf], (it >> 1) & 1, kPolls);
    if (!__syncthreads_and(ok)) {  // (no copy may land later)
      if (t == 0) {
        raise_err(a.err, CSA2_DEVERR_TIMEOUT);
        tc::mbar_wait_bounded(&sy.full[buf], (it >> 1) & 1, kPolls);
        if (item + per < items) tc::mbar_wait_bounded(&sy.full[buf ^ 1], ((it + 1) >> 1) & 1, kPolls);
      }
      break;
    }
    end = last(item + per);
    uint32_t bad = 0;
    float back = 1.0f, fore = 1.0f;
    if constexpr (kNv) {  // a row's largest magnitude: kParts warps
      const uint8_t *mine = st + (warp % kRows) * pitch;
      uint32_t big = 0;
#pragma unroll 4
      for (int c = 16 * (lane + 32 * (warp / kRows)); c < 32 * pieces * kElt; c += 512 * kParts) {
        const uint4 u = *reinterpret_cast<const uint4 *>(mine + c);
        big = word_top<kBf16>(word_top<kBf16>(word_top<kBf16>(word_top<kBf16>(big, u.x), u.y), u.z), u.w);
      }
      if constexpr (kBf16) big = max(big << 16 & 0x7FFF0000u, big & 0x7FFF0000u);
      big = __reduce_max_sync(0xffffffffu, big);
      if (lane == 0) sy.part[warp] = big;
      __syncthreads();
      big = sy.part[r8];
#pragma unroll
      for (int i = 1; i < kParts; ++i) big = max(big, sy.part[r8 + kRows * i]);
      const int e = row_exponent(big, bad);
      back = pow2f(bad ? 0 : -e), fore = pow2f(bad ? 0 : e);
    }
    uint8_t *tiles = a.m.tiles + static_cast<int64_t>(row / kF4Rows) * ct * f4_tile_bytes(kNv);
    const int n8 = t / kRows, turn = kTurns == 3 ? (kBf16 ? n8 >> 1 : n8) & 3 : kTurns == 0 ? 0 : kRows == 4 ? 2 * (n8 & 1) : n8 & 2;
    for (int p = kG * n8; p < pieces && row < rows; p += kG * (kQThreads / kRows))
      put_pieces<kNv, kBf16, kG, kTurns>(tiles, st + r8 * pitch, p, 32 * pieces, m, back, fore, turn, bad);
    if constexpr (!kNv) {  // a bit for each row
      const uint32_t mask = __reduce_or_sync(0xffffffffu, bad ? 1u << r8 : 0u);
      if (lane == 0) sy.part[warp] = mask;
    }
    __syncthreads();  // the buffer has been read
    if (t == 0 && item + 2 * per < items) fetch(item + 2 * per, buf);
    if (t < kRows && row < rows) {
      if constexpr (!kNv) {
        for (int i = 0; i < kQThreads / 32; ++i) bad |= sy.part[i] >> r8 & 1u;
      }
      a.m.row_scales[row] = bad ? __uint_as_float(kNan) : fore;
      if (bad) raise_err(a.err, CSA2_DEVERR_NAN);
    }
  }
}

// A warp: 4 rows of a tile at a time, two groups of rows a time; a lane 16 values of a row in
// chunks that eight lanes store as one run of 128 bytes (bf16: 8 values from 8 u and from 64 +
// 8 u; 32 bytes a lane took 17.8 us for 8,192 x 4,104, whose rows begin in the middle of a
// sector) or of 256 (fp32: 16 values from 16 u).
template <bool kNv, bool kBf16>
__global__ void __launch_bounds__(256) k_fp4_read(csa2_fp4_matrix mx, void *out, int64_t stride, int wide) {
  next_may_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = lane & 7;
  const int ct = static_cast<int>(f4_col_tiles(mx.cols));
  const int row0 = blockIdx.x * 8 + (lane >> 3), m0 = row0 % kF4Rows;  // and row0 + 4, in the same tile
  const uint8_t *tiles = mx.tiles + static_cast<int64_t>(row0 / kF4Rows) * ct * f4_tile_bytes(kNv);
  bool there[2];
  float r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    there[i] = row0 + 4 * i < mx.rows;
    r[i] = there[i] ? mx.row_scales[row0 + 4 * i] : 0.0f;
  }
  for (int k = blockIdx.y * 8 + warp; k < ct; k += 8 * gridDim.y) {
    const uint8_t *rec = tiles + static_cast<int64_t>(k) * f4_tile_bytes(kNv), *sc = rec + kF4CodeBytes;
    uint32_t w[2][2], c[2][2];  // per row and 8 values
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int m = m0 + 4 * i, n = kBf16 ? u + 8 * z : 2 * u + z;  // of the 16 eights of the tile's row
        w[i][z] = there[i] ? load_now(reinterpret_cast<const uint32_t *>(rec + (n >> 2) * 2048 + m * 16 + 4 * (n & 3))) : 0u;
        c[i][z] = there[i] ? (kNv ? sc[512 * (n >> 3) + f4_scale_at(m) + ((n >> 1) & 3)] : sc[f4_scale_at(m) + (n >> 2)]) : 0u;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!there[i]) continue;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int col = kF4Cols * k + 8 * (kBf16 ? u + 8 * z : 2 * u + z);
        const float s = (kNv ? e4m3_value(c[i][z]) : e8m0_value(c[i][z])) * r[i];
        uint32_t h[4];
        e2m1x8_h2(w[i][z], h);
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[q]));
          v[2 * q] = f.x * s;
          v[2 * q + 1] = f.y * s;
        }
        const int64_t at = (row0 + 4 * i) * stride + col;
        if (col + 8 <= mx.cols) {
          if constexpr (kBf16) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
              o[q] = *reinterpret_cast<uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
          } else {
            float *dst = static_cast<float *>(out) + at;
            if (wide) {
              asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                           "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                           : "memory");
            } else {
              reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
              reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (col + q < mx.cols) {
              if constexpr (kBf16) static_cast<__nv_bfloat16 *>(out)[at + q] = __float2bfloat16_rn(v[q]);
              else static_cast<float *>(out)[at + q] = v[q];
            }
        }
      }
    }
  }
}

}  // namespace

template <bool kNv, bool kBf16, bool kStaged>
static cudaError_t launch_rows(const F4Args &a, int pitch, cudaStream_t s) {
  const auto kern = k_fp4_quant_rows<kNv, kBf16, kStaged>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), 8 * pitch);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3((a.m.rows + 7) / 8), kQThreads, 8 * pitch, 0, s, a, pitch);
}
template <bool kNv, bool kBf16, int kRows>
static cudaError_t launch_piped(const F4Args &a, int pitch, cudaStream_t s) {
  const auto kern = k_fp4_quant_piped<kNv, kBf16, kRows>;
  const int bytes = 2 * kRows * pitch, items = (a.m.rows + kRows - 1) / kRows;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), bytes);
  if (e != cudaSuccess) return e;
  const int fit = 227 * 1024 / (bytes + 2048), most = (fit < 3 ? fit : 3) * device_sm_count();
  return launch_after(kern, dim3(items < most ? items : most), kQThreads, bytes, 0, s, a, pitch);
}
// Which kernel.  One GB300, us, in a graph.
//   Up to eight rows per SM a block per row (a block per 8 rows would leave SMs idle).
//   NV, 32 rows per SM and more, as long as four blocks of 8 rows fit an SM: 8,000 x 2,048 bf16
//   7.5 against 8.5 piped, x 2,504 10.1 against 11.3; with fewer rows 2,500 x 512 bf16 3.5
//   against 3.1 piped.
//   Piped, 8 rows at a time while five buffers fit an SM (2,500 x 2,048 bf16 4.5 against 5.4 with
//   4; 1,300 x 4,096 5.9 against 4.5), 4 while two blocks fit (8,000 x 5,120 bf16 20.4 against
//   24.8 with 2, x 7,224 34.6 against 27.7), else 2, or 1, while a block fits: 8,000 x 12,288 fp32 to
//   NV 68 against 159 read through the caches, 5,000 x 20,000 fp32 to NV 79 against 182, to MX
//   76 against 103.
template <bool kNv, bool kBf16>
static cudaError_t launch_quant(const F4Args &a, cudaStream_t s) {
  const int sms = device_sm_count(), rows = a.m.rows;
  if (rows < 8 * sms) {
    const int64_t iter = (f4_col_tiles(a.m.cols) * kF4Cols + 8 * kQThreads - 1) / (8 * kQThreads);
    const auto kern = iter <= 1 ? k_fp4_quant_row<kNv, kBf16, 1> : iter == 2 ? k_fp4_quant_row<kNv, kBf16, 2>
                    : iter == 3 ? k_fp4_quant_row<kNv, kBf16, 3> : k_fp4_quant_row<kNv, kBf16, 4>;
    return launch_after(kern, dim3(rows), kQThreads, 0, 0, s, a);
  }
  constexpr int kK = 1024;
  const int pitch = static_cast<int>(f4_col_tiles(a.m.cols)) * kF4Cols * (kBf16 ? 2 : 4) + 16;
  if constexpr (kNv)
    if (rows >= 32 * sms && 8 * pitch <= 50 * kK) return launch_rows<true, kBf16, true>(a, pitch, s);
  if (rows >= 16 * sms && 8 * pitch <= 40 * kK) return launch_piped<kNv, kBf16, 8>(a, pitch, s);
  if (4 * pitch <= 44 * kK) return launch_piped<kNv, kBf16, 4>(a, pitch, s);
  if (2 * pitch <= 110 * kK) return launch_piped<kNv, kBf16, 2>(a, pitch, s);
  if (pitch <= 110 * kK) return launch_piped<kNv, kBf16, 1>(a, pitch, s);
  return launch_rows<kNv, kBf16, false>(a, 0, s);
}

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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = in_dtype == CSA2_IN_BF16;
  const cudaError_t e = m->format == CSA2_FP4_NV ? (bf ? csa2::launch_quant<true, true>(a, s) : csa2::launch_quant<true, false>(a, s))
                                                 : (bf ? csa2::launch_quant<false, true>(a, s) : csa2::launch_quant<false, false>(a, s));
  return cuda_status(e, "csa2_fp4_quant launch");
}

csa2_status csa2_fp4_read(const csa2_fp4_matrix *m, void *out, int64_t out_stride, int32_t out_dtype, csa2_stream_t stream) {
  csa2_status st = csa2::check_fp4(m, "m");
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(out_dtype == CSA2_OUT_F32 || out_dtype == CSA2_OUT_BF16, CSA2_ERR_RANGE, "out_dtype %d", out_dtype);
  CSA2_REQUIRE(out_stride >= m->cols && out_stride % 8 == 0, CSA2_ERR_SHAPE,
               "out_stride %lld must be a multiple of 8, %d at least", static_cast<long long>(out_stride), m->cols);
  if (m->rows == 0) return CSA2_OK;
  CSA2_REQUIRE_PTR(out);
  const int ct = static_cast<int>(csa2::f4_col_tiles(m->cols)), row_blocks = (m->rows + 7) / 8;
  // a row group's tiles over several blocks: eight per SM in all (2,048 x 4,096 fp32 5.9 us against
  // 8.9 with four), two at least (12,288 x 4,096 21.6 against 23.6 with one)
  int split = 8 * csa2::device_sm_count() / row_blocks;
  split = split < 2 ? 2 : split;
  split = split > (ct + 7) / 8 ? (ct + 7) / 8 : split;
  const int wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  const dim3 grid(row_blocks, split);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = out_dtype == CSA2_OUT_BF16;
  const auto kern = m->format == CSA2_FP4_NV ? (bf ? csa2::k_fp4_read<true, true> : csa2::k_fp4_read<true, false>)
                                             : (bf ? csa2::k_fp4_read<false, true> : csa2::k_fp4_read<false, false>);
  return cuda_status(csa2::launch_after(kern, grid, 256, 0, 0, s, *m, out, out_stride, wide), "csa2_fp4_read launch");
}

}  // extern "C"
