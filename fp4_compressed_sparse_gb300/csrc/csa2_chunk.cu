// csa2_chunk.cu -- dense attention of a ragged batch's new tokens over every
// visible cache entry and the sliding window (csa2_chunk_attn).
//
// z_j = sm_scale q . e_j over 576 dims, o = sum_j p_j c_j over the 512 latent
// dims, p the softmax with an optional sink in its denominator: one pass over
// the keys with a running reference maximum and sum in fp32.
//
// A sequence's query rows (token, head) are cut into row tiles of 64 rows; a
// row tile's keys are the visible entries 0 .. T-1 followed by its window
// tokens, in key tiles of 128 (an entry tile never straddles a page).  Three
// launches: k_chunk_plan lists the row tiles and deals all key tiles out evenly
// over the SMs (a row tile may be shared by several CTAs, at most two partial
// results per CTA), k_chunk_attn computes, k_chunk_merge joins the row tiles
// that were shared.
//
// Work and bound.  2 x 1088 flop per (row, key) against 324 B per key: with 64
// heads 430 flop per byte, so the tensor cores bound it, not HBM.  With 64 rows
// the operands' shared-memory reads (6 KB per 32-cycle MMA step, 128 B per
// cycle) allow about two thirds of the tensor rate.
#include <cmath>
#include <cuda_fp16.h>

#include "csa2_decode.cuh"
#include "csa2_internal.cuh"
#include "csa2_tc.cuh"

namespace csa2 {
namespace {

constexpr int kRows = 64;                        // rows of a row tile
constexpr int kKeys = 128;                       // keys of a key tile
constexpr int kBlk = kKeys * 128;                // one 64-dim block of a key tile: 16 KB
constexpr int kQBlk = kRows * 128;               // one 64-dim block of the query: 8 KB
constexpr int kBlocks = kDqk / 64;               // 9: 8 latent, 1 RoPE
constexpr int kSmWarps = 8, kPrWarps = 8;        // softmax / producer warps
constexpr int kMmaWarp = kSmWarps + kPrWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr uint32_t kColS = 0, kColO = 256;       // TMEM columns: S^T 64, O^T 4 x 64
constexpr uint32_t kWaitIters = 200;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kUnset = -1e30f;                 // reference maximum of a row that has seen no key
constexpr float kTop = 8.0f, kSlack = 15.0f;     // a new reference puts the maximum at 2^8; 2^15 still fits fp16
constexpr int64_t kPartFloats = 4 * 64 * kKeys + 2 * kRows;  // O^T [4][16][128][4], then (m, l) per row

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

// One row tile: rows row0 .. row0 + nrows - 1 of q (flattened token x head).
struct __align__(16) RowTile {
  int64_t row0;
  int64_t pos0;   // position of the first row's token
  int64_t win0;   // row of token pos0 - 127 among the chunk's window rows (used with win_codes)
  int32_t seq;
  int32_t head0;  // the first row's head
  int32_t nrows;
  int32_t T;      // entries its last row sees
  int32_t nkeys;  // T + window tokens
  int32_t ntiles;
  int32_t pad[2];
};
struct CtaRange {
  int64_t lo, hi;  // units [lo, hi) of the whole work (a row tile of n key tiles is n + 1 units)
  int32_t tile;    // the row tile that holds unit lo
  int32_t pad;
};
struct Plan {
  int32_t *seq_tile;  // [batch + 1] first row tile of each sequence
  int64_t *cum;       // [max_tiles + 1] first unit of each row tile
  RowTile *tile;      // [max_tiles]
  CtaRange *cta;      // [n_cta]
  float *part;        // [2 n_cta][kPartFloats]
  int max_tiles, n_cta;
};

__host__ __device__ inline int64_t visible(int64_t pos, int ratio, int64_t cap) {
  const int64_t v = pos > 0 ? pos / ratio : 0;
  return v < cap ? v : cap;
}

// ------------------------------------------------------------------ plan
// Inclusive scan over a 1024-thread block.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += sh[w];
  return v + base;
}

__global__ void __launch_bounds__(1024) k_chunk_plan(ChunkArgs a, Plan p) {
  __shared__ int64_t sh[32];
  __shared__ int64_t carry;
  const int tid = threadIdx.x;
  const csa2_cache &c = a.c;
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int b0 = 0; b0 < c.batch; b0 += 1024) {  // row tiles of each sequence
    const int b = b0 + tid;
    int first = 0, n = 0;
    if (b < c.batch && !ragged_rows(a.cu, b, a.total, a.max_new, first, n)) raise_err(a.err, CSA2_DEVERR_INDEX);
    const int64_t rt = (static_cast<int64_t>(n) * a.heads + kRows - 1) / kRows;
    const int64_t incl = block_scan(rt, sh) + carry;
    if (b < c.batch) p.seq_tile[b + 1] = static_cast<int32_t>(min(incl, static_cast<int64_t>(p.max_tiles)));
    if (b == 0) p.seq_tile[0] = 0;
    __syncthreads();
    if (tid == 1023) carry = incl;
    __syncthreads();
  }
  // overlapping sequences (a broken cu) may ask for more row tiles than there are rows
  if (tid == 0 && carry > p.max_tiles) raise_err(a.err, CSA2_DEVERR_INDEX);
  const int n_tiles = static_cast<int>(min(carry, static_cast<int64_t>(p.max_tiles)));
  __syncthreads();
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int t0 = 0; t0 < n_tiles; t0 += 1024) {
    const int t = t0 + tid;
    int64_t units = 0;
    if (t < n_tiles) {
      int lo = 0, hi = c.batch;  // seq_tile[lo] <= t < seq_tile[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.seq_tile[mid] <= t) lo = mid;
        else hi = mid;
      }
      int first, n;
      ragged_rows(a.cu, lo, a.total, a.max_new, first, n);
      const int64_t r0 = static_cast<int64_t>(t - p.seq_tile[lo]) * kRows;  // within the sequence
      const int64_t left = static_cast<int64_t>(n) * a.heads - r0;
      RowTile x{};
      x.seq = lo;
      x.nrows = static_cast<int>(left < kRows ? left : kRows);
      x.row0 = static_cast<int64_t>(first) * a.heads + r0;
      x.head0 = static_cast<int>(r0 % a.heads);
      const int tok0 = static_cast<int>(r0 / a.heads), tok1 = static_cast<int>((r0 + x.nrows - 1) / a.heads);
      const int64_t P = c.n_tokens[lo] - n;
      x.pos0 = P + tok0;
      x.win0 = static_cast<int64_t>(first) + static_cast<int64_t>(kWin) * lo + tok0 + 1;
      x.T = static_cast<int>(visible(P + tok1, c.ratio, c.capacity));
      x.nkeys = x.T + kWin + (tok1 - tok0);
      x.ntiles = (x.nkeys + kKeys - 1) / kKeys;
      p.tile[t] = x;
      units = x.ntiles + 1;
    }
    const int64_t incl = block_scan(units, sh) + carry;
    if (t < n_tiles) p.cum[t + 1] = incl;
    if (t == 0) p.cum[0] = 0;
    __syncthreads();
    if (tid == 1023) carry = incl;
    __syncthreads();
  }
  const int64_t W = carry;
  // small work on fewer CTAs: two units each at least
  const int64_t g_eff = max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.n_cta), (W + 1) / 2));
  for (int g = tid; g < p.n_cta; g += 1024) {
    CtaRange r{};
    if (g < g_eff) {
      r.lo = W * g / g_eff;
      r.hi = W * (g + 1) / g_eff;
      int lo = 0, hi = n_tiles;  // cum[lo] <= r.lo < cum[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cum[mid] <= r.lo) lo = mid;
        else hi = mid;
      }
      r.tile = lo;
    }
    p.cta[g] = r;
  }
}

// ------------------------------------------------------------------ operands
// Shared-memory matrix descriptor, 128-byte swizzle (atoms of 8 rows x 128 B).
// K-major: lbo unused, sbo between 8-row groups.  MN-major (64 values of M / N
// per 128 B row, one row per k): lbo between 64-value atoms along M / N, sbo
// between groups of 8 k.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// kind::f16, fp16 x fp16 -> fp32; mn: both operands MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, int mn) {
  return (1u << 4) | (static_cast<uint32_t>(mn) << 15) | (static_cast<uint32_t>(mn) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t hmul2u(uint32_t x, uint32_t y) {
  __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&x), *reinterpret_cast<__half2 *>(&y));
  return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t e4m3x2_h2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x2_h2(uint32_t byte) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(r) : "r"(byte));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ uint4 ldg16(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct __align__(1024) ChunkSmem {
  uint8_t k[kBlocks][kBlk];   // the key tile in fp16; block 8 (RoPE) then holds P^T
  uint8_t q[kBlocks][kQBlk];
  __align__(16) float2 fm[kRows];      // logit factor and minus the reference maximum (log2 units) of each row
  __align__(16) float alpha[kRows];
  __align__(16) float fin[kRows];
  __align__(16) float qf[kRows];
  float lsum[4][kRows];
  int32_t rowmax[kRows];               // ordered-int maxima of a tile (reference updates)
  int32_t vis[kRows], w0[kRows];       // a row sees keys j < vis and w0 <= j < w0 + 128
  float sg[2][kKeys];                  // sigma of each key (-inf: no key)
  int plain[2];                        // every key valid with sigma 0
  uint32_t tmem;
  __align__(8) uint64_t full[5];       // dims 128 i .. of the tile filled (4: RoPE)
  __align__(8) uint64_t empty[5];      // ... read by the last MMA (4: P too)
  __align__(8) uint64_t s_full, p_full, q_ready;
};

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, int32_t *err) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    ok = tc::mbar_wait_bounded(bar, parity, kWaitIters) ? 1 : 0;
    if (!ok) raise_err(err, CSA2_DEVERR_TIMEOUT);
  }
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
__device__ __forceinline__ int bar_softmax_or(int v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(v)
      : "memory");
  return r;
}
__device__ __forceinline__ void bar_producers() { asm volatile("bar.sync 2, 256;\n" ::: "memory"); }
__device__ __forceinline__ int32_t order_int(float f) {
  const int32_t i = __float_as_int(f);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float order_float(int32_t i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

// The work items of one CTA, in order: key tiles [k0, k1) of row tile t.
struct Items {
  const Plan &p;
  CtaRange r;
  int t;
  int64_t c0;
  RowTile x;
  int k0, k1;
  __device__ __forceinline__ Items(const Plan &plan, int g) : p(plan), r(plan.cta[g]), t(r.tile - 1), c0(0) {}
  __device__ __forceinline__ bool next() {
    for (;;) {
      ++t;
      if (r.hi <= r.lo) return false;
      c0 = p.cum[t];
      if (c0 >= r.hi || t >= p.max_tiles) return false;
      x = p.tile[t];
      k0 = static_cast<int>(r.lo > c0 ? r.lo - c0 : 0);
      k1 = static_cast<int>(r.hi - c0 < x.ntiles ? r.hi - c0 : x.ntiles);
      if (k0 < k1) return true;
      if (c0 + x.ntiles + 1 >= r.hi) return false;
    }
  }
};

// sigma of a key whose largest magnitude is about 2^e: zero while fp16 holds the
// values as they are, else what brings the largest to about 2^8.
__device__ __forceinline__ int sigma_of(int e) {
  if (e < -1000 || (e >= 0 && e <= 15)) return 0;
  return max(-24, min(120, e - 8));
}

// ------------------------------------------------------------------ producers
// Tiles of whole entries in the common formats come through registers, half a
// tile ahead: step s < 8 is dims 128 (s / 2) .. of keys 64 (s % 2) .., one quarter
// (32 dims) of a key per thread; steps 8, 9 are the RoPE dims.
struct RawFp4 {
  uint4 w;
  uint32_t sc;
};
struct RawFp8 {
  uint4 w[2];
  uint32_t sc;
};
__device__ __forceinline__ void load_raw(const csa2_cache &c, int64_t base, int s, int pt, RawFp4 &r) {
  if (s < 8) {
    const int64_t e = base + 64 * (s & 1) + (pt >> 2);
    r.w = ldg16(c.lat_codes + e * 256 + 64 * (s >> 1) + 16 * (pt & 3));
    r.sc = __ldg(reinterpret_cast<const uint16_t *>(c.lat_scales + e * 32 + 8 * (s >> 1) + 2 * (pt & 3)));
  } else if (s == 8) {
    const int64_t e = base + (pt >> 1);
    r.w = ldg16(c.rope_codes + e * 32 + 16 * (pt & 1));
    r.sc = __ldg(reinterpret_cast<const uint16_t *>(c.rope_scales + e * 4 + 2 * (pt & 1)));
  }
}
__device__ __forceinline__ void load_raw(const csa2_cache &c, int64_t base, int s, int pt, RawFp8 &r) {
  const int64_t e = base + 64 * (s & 1) + (pt >> 2);
  const uint8_t *src = s < 8 ? c.lat_codes + e * 512 + 128 * (s >> 1) + 32 * (pt & 3) : c.rope_codes + e * 128 + 32 * (pt & 3);
  r.w[0] = ldg16(src);
  r.w[1] = ldg16(src + 16);
  if (s < 8) r.sc = __ldg(c.lat_scales + e * 16 + 4 * (s >> 1) + (pt & 3));
}
__device__ __forceinline__ uint4 dq_e2m1(uint32_t w, uint32_t s2) {
  return make_uint4(hmul2u(e2m1x2_h2(w), s2), hmul2u(e2m1x2_h2(w >> 8), s2), hmul2u(e2m1x2_h2(w >> 16), s2),
                    hmul2u(e2m1x2_h2(w >> 24), s2));
}
// 16-byte chunk x (8 dims) of key `key` in a 64-dim block
__device__ __forceinline__ uint8_t *chunk_at(uint8_t *blk, int key, int x) { return blk + key * 128 + ((x ^ (key & 7)) << 4); }

__device__ __forceinline__ void store_raw(ChunkSmem &sm, int s, int pt, const RawFp4 &r, int) {
  uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
  uint32_t sa = e4m3x2_h2((r.sc & 0xFF) * 0x101), sb = e4m3x2_h2((r.sc >> 8) * 0x101);
  if (s < 8) {
    const int key = 64 * (s & 1) + (pt >> 2), qd = pt & 3;
    uint8_t *blk = sm.k[2 * (s >> 1) + (qd >> 1)];
    // the second block's lanes take their chunks in the order 2 3 0 1, so that the
    // eight lanes of a store phase (2 keys x 4 quarters) hit eight different 16 B banks
    const int flip = qd & 2;
    if (flip) {
      const uint32_t t0 = w[0], t1 = w[1], ts = sa;
      w[0] = w[2], w[1] = w[3], w[2] = t0, w[3] = t1, sa = sb, sb = ts;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4 *>(chunk_at(blk, key, 4 * (qd & 1) + (i ^ flip))) = dq_e2m1(w[i], i < 2 ? sa : sb);
  } else if (s == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4 *>(chunk_at(sm.k[8], pt >> 1, 4 * (pt & 1) + i)) = dq_e2m1(w[i], i < 2 ? sa : sb);
  }
}
// factor 2^k as an fp16 pair (k <= 15; zero where fp16 has no such value)
__device__ __forceinline__ uint32_t pow2_h2(int k) {
  const uint32_t h = k < -24 ? 0u : k < -14 ? 1u << (k + 24) : static_cast<uint32_t>(k + 15) << 10;
  return h * 0x10001u;
}
__device__ __forceinline__ void store_raw(ChunkSmem &sm, int s, int pt, const RawFp8 &r, int sigma) {
  const int key = 64 * (s & 1) + (pt >> 2), qd = pt & 3;
  uint32_t o[16];
  const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
  if (s < 8) {
    const uint32_t m2 = pow2_h2(static_cast<int>(r.sc) - 127 - sigma);
    const int flip = qd & 2;
    uint8_t *blk = sm.k[2 * (s >> 1) + (qd >> 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[2 * i] = hmul2u(e4m3x2_h2(w[i]), m2);
      o[2 * i + 1] = hmul2u(e4m3x2_h2(w[i] >> 16), m2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = i ^ 2;
      *reinterpret_cast<uint4 *>(chunk_at(blk, key, 4 * (qd & 1) + (i ^ flip))) =
          flip ? make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3])
               : make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
  } else {  // 16 RoPE dims in bf16
    const float inv = pow2f(-sigma);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = pack_h2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xFFFF0000u) * inv);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4 *>(chunk_at(sm.k[8], key, 2 * qd + i)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
}
template <class Raw>
struct IsFp4 {
  static constexpr bool v = false;
};
template <>
struct IsFp4<RawFp4> {
  static constexpr bool v = true;
};
__device__ __forceinline__ int e8m0_top(uint4 s, int more) {  // largest of 16 scale bytes and `more`
  uint32_t m = __vmaxu4(__vmaxu4(s.x, s.y), __vmaxu4(s.z, s.w));
  m = __vmaxu4(m, m >> 16);
  m = max(m & 0xFF, (m >> 8) & 0xFF);
  return max(static_cast<int>(m), more);
}
__device__ __forceinline__ uint32_t bf16_top(uint4 v, uint32_t m) {  // largest magnitude bits of 8 bf16
  const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
  return __vmaxu2(m, __vmaxu2(a, b));
}
// exponent e (largest magnitude about 2^e) of a key: an E8M0 top (block maximum
// about 2^(top - 119)) and / or the largest bf16 magnitude
__device__ __forceinline__ int key_exponent(int e8, uint32_t bf) {
  const int mb = max(bf & 0xFFFF, bf >> 16);
  const int a = e8 > 0 ? e8 - 119 : -2000, b = mb > 0 ? (mb >> 7) - 127 : -2000;
  return max(a, b);
}

// A tile that is not made of whole entries alone: key j is entry j (j < T), a
// window token, or nothing.  Two threads per key, straight from memory.
struct TailKey {
  int kind;  // 0 nothing, 1 entry, 2 window row
  int64_t at;
  const uint8_t *codes, *scales;
  int sigma;
};
__device__ __noinline__ void tail_key(const ChunkArgs &a, const RowTile &x, int64_t j, int half, TailKey &k) {
  const csa2_cache &c = a.c;
  k.kind = 0;
  k.sigma = 0;
  if (j < x.T) {
    k.at = phys_entry(entry_map(c), x.seq, j);
    if (k.at >= 0) k.kind = 1;
    else raise_err(a.err, CSA2_DEVERR_INDEX);
  } else if (j < x.nkeys) {
    const int64_t tok = x.pos0 - (kWin - 1) + (j - x.T);
    if (tok >= 0) {
      if (a.win_codes != nullptr) {
        k.kind = 2;
        k.codes = a.win_codes;
        k.scales = a.win_scales;
        k.at = x.win0 + (j - x.T);
      } else if (tok >= c.n_tokens[x.seq] - kWin) {
        k.kind = 2;
        k.codes = c.swa_codes;
        k.scales = c.swa_scales;
        k.at = static_cast<int64_t>(x.seq) * kWin + (tok & (kWin - 1));
      } else {
        raise_err(a.err, CSA2_DEVERR_INDEX);
      }
    }
  }
  int e8 = 0;
  uint32_t bf = 0;
  if (k.kind == 1 && c.entry_format == CSA2_ENTRY_FP8) {
    e8 = e8m0_top(*reinterpret_cast<const uint4 *>(c.lat_scales + k.at * 16), 0);
    const uint4 *rc = reinterpret_cast<const uint4 *>(c.rope_codes + k.at * 128);
    for (int i = 4 * half; i < 4 * half + 4; ++i) bf = bf16_top(rc[i], bf);
  } else if (k.kind == 2) {
    if (c.swa_dtype == CSA2_SWA_MXFP8) {
      const uint8_t *s = k.scales + k.at * kSwaScaleStride;
      e8 = e8m0_top(*reinterpret_cast<const uint4 *>(s), max(static_cast<int>(s[16]), static_cast<int>(s[17])));
    } else {
      const uint4 *rc = reinterpret_cast<const uint4 *>(k.codes + k.at * 1152);
      for (int i = 36 * half; i < 36 * half + 36; ++i) bf = bf16_top(rc[i], bf);
    }
  }
  bf = __vmaxu2(bf, __shfl_xor_sync(0xffffffffu, bf, 1));
  if (k.kind == 2 || (k.kind == 1 && c.entry_format == CSA2_ENTRY_FP8)) k.sigma = sigma_of(key_exponent(e8, bf));
}
// units u0 .. u0 + n - 1 (8 dims each) of the key into block `blk`, chunks x0 ..
__device__ __noinline__ void tail_fill(const ChunkArgs &a, const TailKey &k, uint8_t *blk, int key, int u0, int x0, int n) {
  const float inv = pow2f(-k.sigma);
  for (int i = 0; i < n; ++i) {
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (k.kind == 1) entry_unit8(a.c, k.at, u0 + i, v);
    else if (k.kind == 2) window_unit8(k.codes, k.scales, a.c.swa_dtype, k.at, u0 + i, v);
    *reinterpret_cast<uint4 *>(chunk_at(blk, key, x0 + i)) =
        make_uint4(pack_h2(v[0] * inv, v[1] * inv), pack_h2(v[2] * inv, v[3] * inv), pack_h2(v[4] * inv, v[5] * inv),
                   pack_h2(v[6] * inv, v[7] * inv));
  }
}

// Physical entry of the first key of key tile kt, or -1 when the tile is not 128
// whole entries of one valid page.
__device__ __forceinline__ int64_t whole_tile(const csa2_cache &c, const RowTile &x, int kt) {
  if ((kt + 1) * static_cast<int64_t>(kKeys) > x.T) return -1;
  return phys_entry(entry_map(c), x.seq, static_cast<int64_t>(kt) * kKeys);
}

template <class Raw>
__device__ __forceinline__ void produce(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, int pt, int lane) {
  constexpr int kSteps = 10, kAhead = 5;
  const csa2_cache &c = a.c;
  Raw raw[kAhead];
  Items it(p, blockIdx.x);
  bool more = it.next(), dead = false;
  int kt = more ? it.k0 : 0;
  int64_t base = more ? whole_tile(c, it.x, kt) : -1;
  if (base >= 0) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) load_raw(c, base, s, pt, raw[s]);
  }
  for (uint32_t n = 0; more; ++n) {  // n: tiles so far
    const RowTile x = it.x;
    const int cur = kt;
    const int64_t cbase = base;
    // the next tile of this CTA
    if (++kt >= it.k1) {
      more = it.next();
      kt = more ? it.k0 : 0;
    }
    base = more ? whole_tile(c, it.x, kt) : -1;
    const uint32_t par = (n & 1) ^ 1;
    if (cbase >= 0) {
      int sig0 = 0, sig1 = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if ((s & 1) == 0) {
          if (n > 0 && !dead) dead = !wait_warp(&sm.empty[s >> 1], par, a.err);
          if (s == 0) {  // the key scalings of this tile (their last readers are two tiles back)
            if (IsFp4<Raw>::v) {
              if (pt < kKeys) sm.sg[n & 1][pt] = 0.0f;
              if (pt == 0) sm.plain[n & 1] = 1;
            } else {
              const int key = pt >> 1, half = pt & 1;
              const int64_t e = cbase + key;
              uint32_t bf = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) bf = bf16_top(ldg16(c.rope_codes + e * 128 + 64 * half + 16 * i), bf);
              bf = __vmaxu2(bf, __shfl_xor_sync(0xffffffffu, bf, 1));
              const int sg = sigma_of(key_exponent(e8m0_top(ldg16(c.lat_scales + e * 16), 0), bf));
              if (half == 0) sm.sg[n & 1][key] = static_cast<float>(sg);
              if (pt == 0) sm.plain[n & 1] = 0;
              bar_producers();
              sig0 = static_cast<int>(sm.sg[n & 1][pt >> 2]);
              sig1 = static_cast<int>(sm.sg[n & 1][64 + (pt >> 2)]);
            }
          }
        }
        store_raw(sm, s, pt, raw[s % kAhead], (s & 1) ? sig1 : sig0);
        if (s + kAhead < kSteps) load_raw(c, cbase, s + kAhead, pt, raw[s % kAhead]);
        else if (base >= 0) load_raw(c, base, s + kAhead - kSteps, pt, raw[s % kAhead]);
        if (s & 1) {
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.full[s >> 1]);
        }
      }
    } else {
      const int key = pt >> 1, half = pt & 1;
      TailKey k;
      tail_key(a, x, static_cast<int64_t>(cur) * kKeys + key, half, k);
      for (int i = 0; i < 5; ++i) {
        if (n > 0 && !dead) dead = !wait_warp(&sm.empty[i], par, a.err);
        if (i == 0) {
          if (half == 0) sm.sg[n & 1][key] = k.kind ? static_cast<float>(k.sigma) : -INFINITY;
          if (pt == 0) sm.plain[n & 1] = 0;
        }
        if (i < 4) tail_fill(a, k, sm.k[2 * i + half], key, 16 * i + 8 * half, 0, 8);
        else tail_fill(a, k, sm.k[8], key, 64 + 4 * half, 4 * half, 4);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.full[i]);
      }
      if (base >= 0) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s) load_raw(c, base, s, pt, raw[s]);
      }
    }
  }
}

// ------------------------------------------------------------------ softmax warps
// Query rows of the item to fp16 with a power-of-two scale per row, and each
// row's bounds.  Eight rows per warp.
__device__ __forceinline__ void load_query(const ChunkArgs &a, const RowTile &x, ChunkSmem &sm, int warp, int lane) {
  constexpr int kPer = kDqk / 2 / 32;  // 9 words per lane
#pragma unroll 1
  for (int j0 = 0; j0 < kRows / kSmWarps; j0 += 4) {
    uint32_t raw[4][kPer];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = warp * (kRows / kSmWarps) + j0 + j;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q + (x.row0 + r) * kDqk);
#pragma unroll
      for (int i = 0; i < kPer; ++i) raw[j][i] = r < x.nrows ? __ldg(src + lane + 32 * i) : 0u;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = warp * (kRows / kSmWarps) + j0 + j;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = __vmaxu2(m, raw[j][i] & 0x7FFF7FFFu);
      m = max(m & 0xFFFF, m >> 16);
      m = __reduce_max_sync(0xffffffffu, m);
      // |q 2^-ex| < 2^15 (a zero row: any scale)
      const int ex = m ? max(static_cast<int>(m >> 7) - 127 - 14, -110) : 0;
      const float inv = pow2f(-ex);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int d = 2 * (lane + 32 * i);
        *reinterpret_cast<uint32_t *>(chunk_at(sm.q[d >> 6], r, (d & 63) >> 3) + 2 * (d & 7)) =
            pack_h2(__uint_as_float(raw[j][i] << 16) * inv, __uint_as_float(raw[j][i] & 0xFFFF0000u) * inv);
      }
      if (lane == 0) {
        sm.qf[r] = pow2f(ex) * a.sm_scale * kLog2e;
        const int dtok = (x.head0 + min(r, x.nrows - 1)) / a.heads;
        sm.vis[r] = static_cast<int>(visible(x.pos0 + dtok, a.c.ratio, a.c.capacity));
        sm.w0[r] = x.T + dtok;
      }
    }
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(&sm.q_ready);
}

// v[0..31] over the 32 lanes: lane i gets the reduction of v[i]
template <class Op>
__device__ __forceinline__ float warp_columns(float *v, int lane, Op op) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return v[0];
}

__device__ __forceinline__ void softmax(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, uint32_t tmem, int tid) {
  const int warp = tid >> 5, lane = tid & 31, quarter = warp & 3, half = warp >> 2;
  const int key = 32 * quarter + lane;
  const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
  const int c0 = 32 * half;  // this thread's rows c0 .. c0 + 31
  bool dead = false;
  uint32_t n = 0;            // tiles so far
  Items it(p, blockIdx.x);
  bool more = it.next();
  if (more) load_query(a, it.x, sm, warp, lane);
  while (more) {
    const RowTile x = it.x;
    const int k0 = it.k0, k1 = it.k1;
    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.0f;
    bar_softmax();  // qf, vis, w0 of every row written; the last item's fm, fin read
    if (tid < kRows) {
      sm.fm[tid] = make_float2(sm.qf[tid], -kUnset);
      sm.rowmax[tid] = order_int(-INFINITY);
    }
    const int vis_all = sm.vis[0];  // the first row sees least
    bar_softmax();
    for (int kt = k0; kt < k1; ++kt, ++n) {
      if (!dead) dead = !wait_warp(&sm.full[4], n & 1, a.err);  // sg, plain of this tile
      if (!dead) dead = !wait_warp(&sm.s_full, n & 1, a.err);
      tc::tc_fence_after();
      const float sg = sm.sg[n & 1][key];
      const bool fast = sm.plain[n & 1] && (kt + 1) * kKeys <= vis_all;
      const float g = sg == -INFINITY ? 0.0f : ex2(sg);
      const int j = kt * kKeys + key;
      float s[32];
      // exponents of the weighted weights: x = z + sigma - m (log2 units)
      auto exponents = [&]() -> float {
        uint32_t *u = reinterpret_cast<uint32_t *>(s);
        tc::tmem_ld_32x32b_x16(tmem + lane_base + kColS + c0, u);
        tc::tmem_ld_32x32b_x16(tmem + lane_base + kColS + c0 + 16, u + 16);
        tc::tmem_ld_wait_x16(u);
        tc::tmem_ld_wait_x16(u + 16);
        float top = -INFINITY;
        if (fast) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(&sm.fm[c0 + i]);
            s[i] = fmaf(s[i], f.x, f.y);
            s[i + 1] = fmaf(s[i + 1], f.z, f.w);
            top = fmaxf(top, fmaxf(s[i], s[i + 1]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 f = sm.fm[c0 + i];
            const int w0 = sm.w0[c0 + i];
            const bool see = j < sm.vis[c0 + i] || (j >= w0 && j < w0 + kWin);
            s[i] = see ? fmaf(s[i] * g, f.x, sg + f.y) : -INFINITY;
            top = fmaxf(top, s[i]);
          }
        }
        return top;
      };
      const float top = exponents();
      if (bar_softmax_or(top > kSlack)) {
        // some row has no reference yet, or outgrew it: the tile's row maxima
        // (relative to the old reference), new references, O^T and l rescaled
        float v[32];
        // logits without the reference
        {
          uint32_t *u = reinterpret_cast<uint32_t *>(v);
          tc::tmem_ld_32x32b_x16(tmem + lane_base + kColS + c0, u);
          tc::tmem_ld_32x32b_x16(tmem + lane_base + kColS + c0 + 16, u + 16);
          tc::tmem_ld_wait_x16(u);
          tc::tmem_ld_wait_x16(u + 16);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = s[i] == -INFINITY ? -INFINITY : fmaf(v[i] * g, sm.fm[c0 + i].x, sg);
        }
        const float mx = warp_columns(v, lane, [](float x0, float y0) { return fmaxf(x0, y0); });
        atomicMax(&sm.rowmax[c0 + lane], order_int(mx));
        bar_softmax();
        if (tid < kRows) {
          const float m_old = -sm.fm[tid].y, t = order_float(sm.rowmax[tid]);
          float al = 1.0f;
          if (t > m_old + kSlack) {  // kUnset: any logit
            const float m_new = t - kTop;
            al = m_old == kUnset ? 0.0f : ex2(m_old - m_new);
            sm.fm[tid].y = -m_new;
          }
          sm.alpha[tid] = al;
          sm.rowmax[tid] = order_int(-INFINITY);
        }
        bar_softmax();
        if (kt > k0) {  // O^T holds something: PV of the last tile has to be complete
          if (!dead) dead = !wait_warp(&sm.empty[4], (n & 1) ^ 1, a.err);
          tc::tc_fence_after();
#pragma unroll 1
          for (int b = 2 * half; b < 2 * half + 2; ++b)
#pragma unroll 1
            for (int h0 = 0; h0 < kRows; h0 += 16) {
              uint32_t r[16];
              const uint32_t ta = tmem + lane_base + kColO + 64 * b + h0;
              tc::tmem_ld_32x32b_x16(ta, r);
              tc::tmem_ld_wait_x16(r);
#pragma unroll
              for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * sm.alpha[h0 + i]);
              tmem_st_x16(ta, r);
            }
          asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) l[i] *= sm.alpha[c0 + i];
        exponents();
      }
      // weights: l in fp32 (without sigma), P^T to fp16 (with it; at most 2^15)
      const float inv_g = fast ? 1.0f : ex2(-max(sg, -126.0f));
      uint8_t *pb = sm.k[8];
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 8; h += 2) {
          const float p0 = ex2(s[i + h]), p1 = ex2(s[i + h + 1]);
          l[i + h] = fast ? l[i + h] + p0 : fmaf(p0, inv_g, l[i + h]);
          l[i + h + 1] = fast ? l[i + h + 1] + p1 : fmaf(p1, inv_g, l[i + h + 1]);
          w[h / 2] = pack_h2(p0, p1);
        }
        *reinterpret_cast<uint4 *>(chunk_at(pb, key, (c0 + i) >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.p_full);
    }
    // ---- the item's last tile is on its way: sums, the next item's query, then O^T
    const float ls = warp_columns(l, lane, [](float x0, float y0) { return x0 + y0; });
    sm.lsum[quarter][c0 + lane] = ls;
    more = it.next();
    bar_softmax();
    float m = -INFINITY, sum = 0.0f;  // row tid (tid < 64)
    if (tid < kRows) {
      m = -sm.fm[tid].y;
      sum = sm.lsum[0][tid] + sm.lsum[1][tid] + sm.lsum[2][tid] + sm.lsum[3][tid];
      if (m == kUnset) m = -INFINITY;
    }
    const bool direct = k0 == 0 && k1 == x.ntiles;
    if (tid < kRows && direct) {
      float f = 1.0f;
      if (a.sink != nullptr) {
        const float z = a.sink[(x.head0 + tid) % a.heads] * kLog2e;
        const float mf = fmaxf(m, z);
        f = m == -INFINITY ? 0.0f : ex2(m - mf);
        sum = sum * f + ex2(z - mf);
        m = mf;
      }
      sm.fin[tid] = sum > 0.0f ? f / sum : 0.0f;
      if (tid < x.nrows) a.lse[x.row0 + tid] = sum > 0.0f ? (m + log2f(sum)) * kLn2 : -INFINITY;
    }
    if (more) load_query(a, it.x, sm, warp, lane);
    bar_softmax();  // fin written
    if (!dead) dead = !wait_warp(&sm.empty[4], (n - 1) & 1, a.err);  // PV of the last tile
    tc::tc_fence_after();
    const int slot = 2 * blockIdx.x + (k0 > 0 ? 0 : 1);
    float *part = p.part + slot * kPartFloats;
    if (!direct && tid < kRows)
      *reinterpret_cast<float2 *>(part + 4 * 64 * kKeys + 2 * tid) = make_float2(m, sum);
#pragma unroll 1
    for (int b = 2 * half; b < 2 * half + 2; ++b) {
#pragma unroll 1
      for (int h0 = 0; h0 < kRows; h0 += 32) {
        uint32_t r[32];
        tc::tmem_ld_32x32b_x16(tmem + lane_base + kColO + 64 * b + h0, r);
        tc::tmem_ld_32x32b_x16(tmem + lane_base + kColO + 64 * b + h0 + 16, r + 16);
        tc::tmem_ld_wait_x16(r);
        tc::tmem_ld_wait_x16(r + 16);
        if (dead) continue;
        if (!direct) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4 *>(part + ((b * 16 + (h0 + i) / 4) * kKeys + key) * 4) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        } else if (a.bf16) {
          // lane pairs exchange so that each stores two neighbouring dims of one row
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float v0 = __uint_as_float(r[i]) * sm.fin[h0 + i], v1 = __uint_as_float(r[i + 1]) * sm.fin[h0 + i + 1];
            const float o = __shfl_xor_sync(0xffffffffu, lane & 1 ? v0 : v1, 1);
            const int row = h0 + i + (lane & 1);
            const __nv_bfloat162 t2 = lane & 1 ? __floats2bfloat162_rn(o, v1) : __floats2bfloat162_rn(v0, o);
            if (row < x.nrows)
              *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + (x.row0 + row) * kLat + 128 * b + (key & ~1)) = t2;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (h0 + i < x.nrows)
              static_cast<float *>(a.out)[(x.row0 + h0 + i) * kLat + 128 * b + key] = __uint_as_float(r[i]) * sm.fin[h0 + i];
        }
      }
    }
    tc::tc_fence_before();
  }
}

// ------------------------------------------------------------------ MMA issuer
// Per key tile: S^T[128 keys][64 rows] = K Q^T as the tile's dims arrive, then,
// with P^T, O^T[512 dims][64 rows] += V^T P^T in four blocks of 128 dims, each
// handed back to the producers as it completes.
__device__ __forceinline__ void issue(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, uint32_t tmem) {
  constexpr uint32_t idS = idesc_f16(kKeys, kRows, 0), idO = idesc_f16(128, kRows, 1);
  const uint32_t ka = tc::smem_addr(sm.k), qa = tc::smem_addr(sm.q), pa = ka + 8 * kBlk;
  Items it(p, blockIdx.x);
  bool dead = false;
  uint32_t n = 0, items = 0;
  auto wait = [&](uint64_t *bar, uint32_t par) {
    if (!dead && !tc::mbar_wait_bounded(bar, par, kWaitIters)) {
      dead = true;
      raise_err(a.err, CSA2_DEVERR_TIMEOUT);
    }
  };
  while (it.next()) {
    wait(&sm.q_ready, items & 1);
    ++items;
    for (int kt = it.k0; kt < it.k1; ++kt, ++n) {
#pragma unroll 1
      for (int i = 0; i < 5; ++i) {
        wait(&sm.full[i], n & 1);
        if (dead) break;
        tc::tc_fence_after();
        for (int b = 2 * i; b < min(2 * i + 2, kBlocks); ++b)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16(tmem + kColS, desc_sw128(ka + b * kBlk + 32 * kk, 16, 1024), desc_sw128(qa + b * kQBlk + 32 * kk, 16, 1024),
                    idS, (b | kk) ? 1u : 0u);
      }
      if (!dead) tc::mma_commit(&sm.s_full);
      wait(&sm.p_full, n & 1);
      if (dead) break;
      tc::tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16(tmem + kColO + 64 * i, desc_sw128(ka + 2 * i * kBlk + 2048 * ks, kBlk, 1024),
                  desc_sw128(pa + 2048 * ks, kBlk, 1024), idO, (kt > it.k0 || ks) ? 1u : 0u);
        tc::mma_commit(&sm.empty[i]);
      }
      tc::mma_commit(&sm.empty[4]);
    }
    if (dead) break;
  }
}

__global__ void __launch_bounds__(kThreads, 1) k_chunk_attn(ChunkArgs a, Plan p) {
  extern __shared__ uint8_t smem_raw[];
  ChunkSmem &sm = *reinterpret_cast<ChunkSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CtaRange r = p.cta[blockIdx.x];
  if (r.hi <= r.lo) return;  // the whole CTA
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) {
      tc::mbar_init(&sm.full[i], kPrWarps);
      tc::mbar_init(&sm.empty[i], 1);
    }
    tc::mbar_init(&sm.s_full, 1);
    tc::mbar_init(&sm.p_full, kSmWarps);
    tc::mbar_init(&sm.q_ready, kSmWarps);
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp < kSmWarps) {
    softmax(a, p, sm, tmem, tid);
  } else if (warp < kMmaWarp) {
    if (a.c.entry_format == CSA2_ENTRY_FP8) produce<RawFp8>(a, p, sm, tid - 32 * kSmWarps, lane);
    else produce<RawFp4>(a, p, sm, tid - 32 * kSmWarps, lane);
  } else if (lane == 0) {
    issue(a, p, sm, tmem);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Row tiles shared by several CTAs: block (g, y) joins the one that ends in CTA
// g, rows 4 (y % 16) .. of dims 128 (y / 16) .., its parts in CTA order.
__global__ void __launch_bounds__(kKeys) k_chunk_merge(ChunkArgs a, Plan p) {
  const int g = blockIdx.x, blk = blockIdx.y / 16, i4 = blockIdx.y % 16, d = threadIdx.x;
  Items it(p, g);
  if (!it.next() || it.k0 == 0 || it.k1 != it.x.ntiles) return;
  const RowTile &x = it.x;
  if (4 * i4 >= x.nrows) return;
  int g0 = g;  // the CTA that holds the row tile's first key tile
  while (g0 > 0 && p.cta[g0].lo > it.c0) --g0;
  float m[4], l[4], o[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = 0.0f, o[r] = 0.0f;
  for (int k = g0; k <= g; ++k) {  // the reference of the whole row
    const float *ml = p.part + (2 * k + (k == g0 ? 1 : 0)) * kPartFloats + 4 * 64 * kKeys + 8 * i4;
#pragma unroll
    for (int r = 0; r < 4; ++r) m[r] = fmaxf(m[r], ml[2 * r]);
  }
  for (int k = g0; k <= g; ++k) {
    const float *part = p.part + (2 * k + (k == g0 ? 1 : 0)) * kPartFloats, *ml = part + 4 * 64 * kKeys + 8 * i4;
    const float4 v = *reinterpret_cast<const float4 *>(part + ((blk * 16 + i4) * kKeys + d) * 4);
    const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float w = ml[2 * r] == -INFINITY ? 0.0f : ex2(ml[2 * r] - m[r]);
      l[r] = fmaf(w, ml[2 * r + 1], l[r]);
      o[r] = w == 0.0f ? o[r] : fmaf(w, vv[r], o[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * i4 + r;
    if (row >= x.nrows) break;
    float f = 1.0f;
    if (a.sink != nullptr) {
      const float z = a.sink[(x.head0 + row) % a.heads] * kLog2e, mf = fmaxf(m[r], z);
      f = m[r] == -INFINITY ? 0.0f : ex2(m[r] - mf);
      l[r] = l[r] * f + ex2(z - mf);
      m[r] = mf;
    }
    const float v = l[r] > 0.0f ? o[r] * (f / l[r]) : 0.0f;
    const int64_t at = (x.row0 + row) * kLat + 128 * blk + d;
    if (a.bf16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(a.out)[at] = v;
    if (d == 0 && blk == 0) a.lse[x.row0 + row] = l[r] > 0.0f ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
  }
}

struct PlanLayout {
  size_t seq_tile, cum, tile, cta, part, total;
  int max_tiles, n_cta;
};
PlanLayout plan_layout(int batch, int total, int heads) {
  PlanLayout L{};
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  const int64_t t = static_cast<int64_t>(total) * heads / kRows + (batch < total ? batch : total) + 1;
  L.max_tiles = static_cast<int>(t);
  L.n_cta = device_sm_count();
  size_t o = 0;
  L.seq_tile = o;
  o = up(o + (static_cast<size_t>(batch) + 1) * 4);
  L.cum = o;
  o = up(o + (static_cast<size_t>(t) + 1) * 8);
  L.tile = o;
  o = up(o + static_cast<size_t>(t) * sizeof(RowTile));
  L.cta = o;
  o = up(o + static_cast<size_t>(L.n_cta) * sizeof(CtaRange));
  L.part = o;
  o = up(o + static_cast<size_t>(2) * L.n_cta * kPartFloats * 4);
  L.total = o;
  return L;
}

}  // namespace
}  // namespace csa2

extern "C" {

size_t csa2_chunk_attn_workspace_size(int32_t batch, int32_t total, int32_t n_heads) {
  if (batch <= 0 || total <= 0 || n_heads <= 0) return 256;
  return csa2::plan_layout(batch, total, n_heads).total;
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
  const csa2::PlanLayout L = csa2::plan_layout(cache->batch, total, n_heads);
  uint8_t *wb = static_cast<uint8_t *>(ws);
  csa2::Plan p{reinterpret_cast<int32_t *>(wb + L.seq_tile), reinterpret_cast<int64_t *>(wb + L.cum),
               reinterpret_cast<csa2::RowTile *>(wb + L.tile), reinterpret_cast<csa2::CtaRange *>(wb + L.cta),
               reinterpret_cast<float *>(wb + L.part), L.max_tiles, L.n_cta};
  const int smem = static_cast<int>(sizeof(csa2::ChunkSmem)) + 1024;
  static_assert(sizeof(csa2::ChunkSmem) + 1024 <= 232448, "shared memory of one CTA");
  cudaError_t e = csa2::ensure_smem_limit(reinterpret_cast<const void *>(&csa2::k_chunk_attn), smem);
  if (e != cudaSuccess) return cuda_status(e, "csa2_chunk_attn shared memory");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  csa2::k_chunk_plan<<<1, 1024, 0, s>>>(a, p);
  csa2::k_chunk_attn<<<L.n_cta, csa2::kThreads, smem, s>>>(a, p);
  csa2::k_chunk_merge<<<dim3(L.n_cta, 64), csa2::kKeys, 0, s>>>(a, p);
  return cuda_status(cudaGetLastError(), "csa2_chunk_attn launch");
}

}  // extern "C"
