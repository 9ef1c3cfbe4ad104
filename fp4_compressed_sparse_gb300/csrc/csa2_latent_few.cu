// csa2_latent_few.cu -- csa2_query_latent and csa2_value_project for few tokens.
//
// The weights' bytes bound these (8.4 MB for 64 heads of 128: 1.2 us), and before them the
// chain launch -> loads -> products -> sums -> stores.  So all loads of a block's operands
// are issued at once (a query row's position, which decides whether it is stored, is read
// behind the sums): a warp takes W from global memory straight into the fragments of
// mma.sync m16n8k16 (tokens are its 16 rows), 16 bytes a lane, whose values are dealt to
// fragment places by renaming columns (query) or summation indices (value).  The warps of
// a block share out K and join their sums in shared memory, in order.
//
// Measured (in a graph, W in L2): queries of 64 heads of 128, one token 3.9 us, 32 tokens 5.1;
// values, one token 2.9 (bf16) and 3.4 us (fp32), 32 tokens 3.7 and 4.7.  A launch alone takes
// 1.4.  With each call's W in HBM 4.5 and 5.6, 4.0 and 4.4, 4.5 and 5.6; with all else there
// too 7.3 us (queries, one token) and 9.8 us (32 fp32 tokens).
#include "csa2_latent.cuh"

namespace csa2 {
namespace {

constexpr int kFewThreads = 256;

// D[16 tokens][8 columns] += A[16][16] B[16][8]
__device__ __forceinline__ void mma16816(float4 &d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d.x), "+f"(d.y), "+f"(d.z), "+f"(d.w)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Grid (heads, 512 / 128 + 1, groups of 16 kTiles tokens); the last of y rotates the RoPE
// dims.  Warp w: columns 64 (w % 2) .. of the part, K steps w / 2 and w / 2 + 4.  In a
// step a lane (g = lane / 4, t = lane % 4) loads columns 8 g .. 8 g + 7 of the four K rows
// that its fragments hold; column 8 g + v is column g of the v-th product, so its sums
// are of columns 16 t + v and 16 t + 8 + v: 16 in a row.
template <int kTiles>
__global__ void __launch_bounds__(kFewThreads) k_query_few(LatentArgs a) {
  __shared__ float4 red[3][2][kTiles * 8][32];
  next_may_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x, part = blockIdx.y, tok0 = blockIdx.z * 16 * kTiles;
  const uint16_t *xh = static_cast<const uint16_t *>(a.x) + static_cast<int64_t>(h) * (a.dim + kRope);
  if (part == kLat / 128) {
    for (int i = threadIdx.x; i < 16 * kTiles * 8; i += kFewThreads) {
      const int64_t tok = tok0 + i / 8;
      int64_t p;
      if (tok < a.total && row_position(a, tok, h == 0 && i % 8 == 0, p))
        store_rope8(load_rope8(a, xh + tok * a.x_stride + a.dim + 8 * (i % 8), p, i % 8),
                    a.out + tok * a.out_stride + static_cast<int64_t>(h) * kDqk + kLat + 8 * (i % 8));
    }
    return;
  }
  const int cg = warp & 1, ks = warp >> 1, steps = a.dim / 16;
  const uint16_t *w = a.w + h * a.w_stride + part * 128 + cg * 64 + 8 * g;
  uint4 r[2][4];
  uint32_t f[2][kTiles][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = 16 * (ks + 4 * i) + 2 * t;
    const bool there = ks + 4 * i < steps;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[i][j] = there ? load_now(reinterpret_cast<const uint4 *>(w + static_cast<int64_t>(k + (j & 1) + 8 * (j >> 1)) * kLat))
                      : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t tok = tok0 + 16 * m + g + 8 * (j & 1);
        f[i][m][j] = there && tok < a.total ? load_now(reinterpret_cast<const uint32_t *>(xh + tok * a.x_stride + k + 8 * (j >> 1))) : 0u;
      }
  }
  float4 acc[kTiles][8] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const uint32_t sel = v & 1 ? 0x7632 : 0x5410;
      const uint32_t b0 = __byte_perm(word(r[i][0], v >> 1), word(r[i][1], v >> 1), sel);
      const uint32_t b1 = __byte_perm(word(r[i][2], v >> 1), word(r[i][3], v >> 1), sel);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) mma16816(acc[m][v], f[i][m], b0, b1);
    }
  if (ks > 0) {
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int v = 0; v < 8; ++v) red[ks - 1][cg][8 * m + v][lane] = acc[m][v];
  }
  __syncthreads();
  if (ks > 0) return;
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int v = 0; v < 8; ++v)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const float4 o = red[i][cg][8 * m + v][lane];
        acc[m][v].x += o.x;
        acc[m][v].y += o.y;
        acc[m][v].z += o.z;
        acc[m][v].w += o.w;
      }
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t tok = tok0 + 16 * m + g + 8 * half;
      int64_t p;
      if (tok >= a.total || !row_position(a, tok, false, p)) continue;
      uint32_t o[8];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float4 lo = acc[m][2 * v], hi = acc[m][2 * v + 1];
        o[v] = half ? pack_bf16(lo.z, hi.z) : pack_bf16(lo.x, hi.x);
        o[4 + v] = half ? pack_bf16(lo.w, hi.w) : pack_bf16(lo.y, hi.y);
      }
      uint4 *dst = reinterpret_cast<uint4 *>(a.out + tok * a.out_stride + static_cast<int64_t>(h) * kDqk + part * 128 + cg * 64 + 16 * t);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Grid (heads, parts of 32 values, groups of 16 kTiles tokens).  Warp w: latent dims
// 64 w .. 64 w + 63, in two blocks of 32.  In a block a lane loads dims 8 t .. 8 t + 7 of
// row 4 g + v of W for the v-th product, and of its tokens: values 0-3 are its places of
// one K step of 16, values 4-7 of the next, on both sides.  Its sums are of values 8 t + v
// and 8 t + 4 + v: 8 in a row.
template <int kTiles, bool kF32>
__global__ void __launch_bounds__(kFewThreads) k_value_few(LatentArgs a) {
  __shared__ float2 red[8][kTiles][2][4][32];
  next_may_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x, j0 = blockIdx.y * 32, tok0 = blockIdx.z * 16 * kTiles;
  const int c0 = 64 * warp + 8 * t;
  const uint16_t *w = a.w + h * a.w_stride + c0;
  constexpr int kWords = kF32 ? 2 : 1;  // of 16 bytes, for 8 values
  uint4 r[2][4], x[2][kTiles][2][kWords];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int j = j0 + 4 * g + v;
      r[i][v] = j < a.dim ? load_now(reinterpret_cast<const uint4 *>(w + static_cast<int64_t>(j) * kLat + 32 * i)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t tok = tok0 + 16 * m + g + 8 * half;
        const int64_t at = tok * a.x_stride + static_cast<int64_t>(h) * kLat + c0 + 32 * i;
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.x) + at * (kF32 ? 4 : 2));
#pragma unroll
        for (int z = 0; z < kWords; ++z) x[i][m][half][z] = tok < a.total ? load_now(p + z) : make_uint4(0, 0, 0, 0);
      }
  }
  // values 4 s .. 4 s + 3 of two tokens: the MMA's rows, of fp32 latents in three parts (cut
  // before the first product: 32 tokens of 64 heads 4.6 us, cut between products 4.9)
  constexpr int kParts = kF32 ? 3 : 1;
  uint32_t f[2][2][kTiles][kParts][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (kF32) {
            const uint4 &u = x[i][m][j & 1][s];
            uint32_t p[3];
            split3(__uint_as_float(j < 2 ? u.x : u.z), __uint_as_float(j < 2 ? u.y : u.w), p);
#pragma unroll
            for (int z = 0; z < 3; ++z) f[i][s][m][z][j] = p[z];
          } else {
            f[i][s][m][0][j] = word(x[i][m][j & 1][0], 2 * s + (j >> 1));
          }
        }
  float4 acc[kTiles][4] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int z = 0; z < kParts; ++z)
#pragma unroll
          for (int v = 0; v < 4; ++v) mma16816(acc[m][v], f[i][s][m][z], word(r[i][v], 2 * s), word(r[i][v], 2 * s + 1));
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      red[warp][m][0][v][lane] = make_float2(acc[m][v].x, acc[m][v].y);
      red[warp][m][1][v][lane] = make_float2(acc[m][v].z, acc[m][v].w);
    }
  __syncthreads();
  if (warp >= 2 * kTiles) return;
  const int m = warp >> 1, half = warp & 1;
  float2 o[4] = {};
#pragma unroll
  for (int v = 0; v < 4; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = red[i][m][half][v][lane];
      o[v].x += p.x;
      o[v].y += p.y;
    }
  const int64_t tok = tok0 + 16 * m + g + 8 * half;
  const int j = j0 + 8 * t;
  if (tok < a.total && j < a.dim)  // (dim is a multiple of 16)
    *reinterpret_cast<uint4 *>(a.out + tok * a.out_stride + static_cast<int64_t>(h) * a.dim + j) =
        make_uint4(pack_bf16(o[0].x, o[1].x), pack_bf16(o[2].x, o[3].x), pack_bf16(o[0].y, o[1].y), pack_bf16(o[2].y, o[3].y));
}

}  // namespace

cudaError_t launch_query_few(const LatentArgs &a, cudaStream_t s) {
  const dim3 grid(a.heads, kLat / 128 + 1, (a.total + 31) / 32);
  return launch_after(a.total <= 16 ? k_query_few<1> : k_query_few<2>, grid, kFewThreads, 0, 0, s, a);
}

cudaError_t launch_value_few(const LatentArgs &a, bool f32, cudaStream_t s) {
  const dim3 grid(a.heads, (a.dim + 31) / 32, (a.total + 31) / 32);
  const auto kern = a.total <= 16 ? (f32 ? k_value_few<1, true> : k_value_few<1, false>) : (f32 ? k_value_few<2, true> : k_value_few<2, false>);
  return launch_after(kern, grid, kFewThreads, 0, 0, s, a);
}

}  // namespace csa2
