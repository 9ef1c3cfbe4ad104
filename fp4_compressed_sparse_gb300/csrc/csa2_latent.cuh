// csa2_latent.cuh -- what the kernels of csa2_query_latent and csa2_value_project share.
#pragma once

#include "csa2_internal.cuh"

namespace csa2 {

struct LatentArgs {
  const void *x;        // query: bf16 rows of heads x (dim + 64); value: [total][heads][512]
  int64_t x_stride;     // elements per token
  const uint16_t *w;    // head h: rows of 512 at w + h * w_stride
  int64_t w_stride;
  int heads, dim, total;
  const int64_t *pos;   // query
  const float *rope;
  int64_t rope_len;
  uint16_t *out;
  int64_t out_stride;   // elements per token
  int parts;            // column parts of a head
  int np;               // columns of a part
  int halves;           // queries: a CTA's run may begin and end with half a unit
  int tiles;            // token tiles
  int wide;             // 32-byte stores are aligned
  int32_t *err;
};

// Where the forms for few tokens are taken.  One GB300, us, few / persistent, dim 128 (queries
// were swept at that width and at 64, which moves them little):
//   queries of 64 heads, 32 tokens 5.0 / 5.0, 33 tokens 7.4 / 5.0; of 32 heads, 17 tokens 4.1 /
//   3.8, 32 tokens 4.7 / 3.9; of 128 heads, one token 5.6 / 6.1, 5 tokens 5.8 / 5.9, 16 tokens
//   6.8 / 6.0; of 64 heads of 64, 32 tokens 4.0 / 4.4, 33 tokens 6.2 / 4.4;
//   values of 64 heads, 32 tokens bf16 3.7 / 4.1, fp32 4.6 / 8.1, 33 tokens 4.8 / 4.1 and 7.7 /
//   8.1, 65 tokens 5.6 / 4.1 and 10.8 / 8.1; of 128 heads, 16 tokens 3.7 / 4.6 and 5.0 / 8.9, 32
//   tokens 5.2 / 4.6 and 8.1 / 8.8, 33 tokens 7.1 / 4.7 and 12.6 / 9.0; of 16 heads, 129 tokens 3.8 /
//   3.9 and 6.1 / 7.5, 256 tokens 5.1 / 4.0 and 8.2 / 7.6; of 64 heads of 64, 64 tokens 3.7 / 3.8
//   and 4.6 / 7.6.
inline bool few_queries(int total, int heads) { return total <= (heads <= 64 ? 32 : 4); }
// (a block takes 16 or 32 tokens, a head, 32 values)
inline bool few_values(int total, int heads, int dim, bool f32) {
  return static_cast<int64_t>((total + 15) / 16) * heads * ((dim + 31) / 32) <= (f32 ? 768 : 512);
}
cudaError_t launch_query_few(const LatentArgs &a, cudaStream_t s);
cudaError_t launch_value_few(const LatentArgs &a, bool f32, cudaStream_t s);

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
// Two fp32 values as three bf16 parts each (a's in the low half): 8 bits are cut off at a time,
// so that nothing is rounded, a finite value never becomes infinite, and the parts add up to the
// value but for its bits below bf16's least, 2^-133.  An infinity lies in the first part alone; a
// NaN is at least one part's.
__device__ __forceinline__ void split3(float a, float b, uint32_t *part) {
  part[0] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  const float ha = __uint_as_float(part[0] << 16), hb = __uint_as_float(part[0] & 0xFFFF0000u);
  a = a == ha ? 0.0f : a - ha;  // (an infinity less itself would be a NaN)
  b = b == hb ? 0.0f : b - hb;
  part[1] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  a -= __uint_as_float(part[1] << 16);
  b -= __uint_as_float(part[1] & 0xFFFF0000u);
  part[2] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// Whether a query row is written; one behind the RoPE table raises the bit.
__device__ __forceinline__ bool row_position(const LatentArgs &a, int64_t tok, bool report, int64_t &p) {
  p = a.pos[tok];
  if (p >= a.rope_len && report) raise_err(a.err, CSA2_DEVERR_ROPE);
  return p >= 0 && p < a.rope_len;
}
// RoPE dims 8 d8 .. of a head at src, and the table's row of position p.
struct Rope8 {
  uint4 v;
  float4 c0, c1;
};
__device__ __forceinline__ Rope8 load_rope8(const LatentArgs &a, const uint16_t *src, int64_t p, int d8) {
  const float4 *cs = reinterpret_cast<const float4 *>(a.rope + p * kRope + 8 * d8);
  return Rope8{load_now(reinterpret_cast<const uint4 *>(src)), load_now(cs), load_now(cs + 1)};
}
__device__ __forceinline__ void store_rope8(const Rope8 &r, uint16_t *dst) {
  const uint32_t in[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
  const float cc[8] = {r.c0.x, r.c0.y, r.c0.z, r.c0.w, r.c1.x, r.c1.y, r.c1.z, r.c1.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x = __uint_as_float(in[j] << 16), y = __uint_as_float(in[j] & 0xFFFF0000u);
    rope_pair(x, y, cc[2 * j], cc[2 * j + 1]);
    o[j] = pack_bf16(x, y);
  }
  *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace csa2
