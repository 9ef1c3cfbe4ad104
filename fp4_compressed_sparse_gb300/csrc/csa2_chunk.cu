// csa2_chunk.cu -- dense attention of a ragged batch's new tokens over every
// visible cache entry and the sliding window (csa2_chunk_attn).
//
// z_j = sm_scale q . e_j over 576 dims, o = sum_j p_j c_j over the 512 latent
// dims, p the softmax with an optional sink in its denominator: one pass over
// the keys with a running reference maximum and sum in fp32.
//
// A sequence's query rows (token, head) are cut into row tiles of 64 rows; a
// row tile's keys are the visible entries 0 .. T-1 followed by its window
// tokens, in key tiles of 64 (an entry tile never straddles a page).  Three
// launches: k_chunk_plan lists the row tiles and deals all key tiles out evenly
// over the SMs (a row tile may be shared by several CTAs, at most two partial
// results per CTA), k_chunk_attn computes, k_chunk_merge joins the row tiles
// that were shared.
//
// Work and bound.  2 x 1088 flop per (row, key) against 324 B per key: with 64
// heads 430 flop per byte, so the tensor cores bound it, not HBM.
//
// Precision.  S, the sums and O^T are fp32, the operands fp16.  FP4 records are exact
// (E2M1 x E4M3: 6 significant bits, 2^-10 to 2688).  The values of V4 entries and of
// window tokens go in divided by a power of two s per key, 1 where the key's largest
// magnitude is 2^0 to 2^16 (sigma_of): fp16's step there makes them off by 2^-25 s.  The
// weights p, times s, are rounded to fp16 as well, as the MMA takes both operands in
// one type: by 2^-11 of themselves (a bf16 output's rounding is 2^-8), and below
// 2^-14 on a scale on which a row's largest is 2^4 at least by 2^-29 of that.
//
// Tiles.  O^T of 64 rows is 256 columns of tensor memory beside two S; 128 rows
// would take all 512 and leave none for S.  Beside the query (72 KB) two key
// tiles of 64 fit into shared memory (72 KB each), a third does not.
//
// What bounds it now: a key tile's way through its buffer, in cycles about: fill
// 1,650, hand-over 360, QK 1,570 (the MMAs alone 1,177), softmax 1,300 (2,100 when a
// row's reference moves), hand-over 450, PV 880, hand-over 440.  Two buffers make
// that 3,500 to 3,700 per tile; the MMAs by themselves take 1,957 (operands from
// shared memory at 128 B per cycle), the fill's stores 576 more of the same
// bandwidth, so what overlaps also slows each other down.  Tensor pipe 35 %, ALU
// 36 %, issue slots 37 %.
// Measured: 1,024 queries of 64 heads over 15,000 V4 entries 3.53 ms (632 TFLOP/s,
// 33 % of the measured bf16 rate); ragged chunks over FP4 entries 1.34 ms (570);
// 32 single tokens over 8K entries each 94 us, 16 over up to 65K 154 us (504); one
// over 1,000 24 us, of which the three launches' round trips are nearly all.
#include <atomic>
#include <cmath>
#include <cuda_fp16.h>

#include "csa2_decode.cuh"
#include "csa2_internal.cuh"
#include "csa2_tc.cuh"

namespace csa2 {
namespace {

constexpr int kRows = 64;                    // rows of a row tile
constexpr int kKeys = 64;                    // keys of a key tile
constexpr int kBlk = kKeys * 128;            // a 64-dim block of a key tile, or of the query: 8 KB
constexpr int kBlocks = kDqk / 64;           // 9: 8 latent, 1 RoPE
constexpr int kTile = kBlocks * kBlk;        // 73,728 B
constexpr int kSmWarps = 8, kPrWarps = 16;   // softmax / producer warps
constexpr int kMmaWarp = kSmWarps + kPrWarps, kAheadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kAheadWarp + 3);  // whole warpgroups: 2 softmax, 4 producers, 1 that issues
// Registers per thread: 7 x 72 at the launch, then moved from the issuing
// warpgroup to the others (spills in their loops cost 6 to 11 % of the time).
constexpr int kLaunchRegs = 72, kWorkRegs = 80, kIssueRegs = 24;
static_assert(6 * kWorkRegs + kIssueRegs <= 7 * kLaunchRegs, "setmaxnreg draws on the launch's registers");
static_assert(kPrWarps == 16, "plain is read as 16 bytes");
constexpr int kAhead = 4;                    // key tiles requested into L2 ahead of use
constexpr uint32_t kColS = 0, kColO = 256;   // TMEM columns: S 2 x 64, O^T 4 x 64
constexpr uint32_t kWaitIters = 200, kPolls = 1u << 20;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kTop = 4.0f, kSlack = 15.0f;  // a new reference puts the maximum at 2^4; 2^15 still fits fp16
constexpr int64_t kPartFloats = kLat * kRows + 2 * kRows;  // O^T [4][16][128][4], then (m, l) per row

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
  int4 *merge;        // [n_cta] the CTAs in which a shared row tile ends, with its first CTA and its index; then -1
  float *part;        // [2 n_cta][kPartFloats]
  int max_tiles, n_cta;
};

__host__ __device__ inline int64_t visible(int64_t pos, int ratio, int64_t cap) {
  const int64_t v = pos > 0 ? pos >> (ratio - 1) : 0;  // ratio 1 or 2
  return v < cap ? v : cap;
}

// ------------------------------------------------------------------ plan
// Inclusive scan over the block.
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
  int64_t w = warp > lane ? sh[lane] : 0;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return v + w;
}
// Largest i in [0, n) with list[i] <= v (list[0] <= v): a binary search.
template <class T>
__device__ __forceinline__ int last_at_most(const T *list, int n, T v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One block: 5 us for decode batches, 10 us for a thousand row tiles, 64 us for 16,384
// (lists too long for shared memory; the attention of those then takes 26 ms).  The two
// lists it searches (first row tile of each sequence, first unit of each row tile)
// are kept in shared memory as far as they fit, as a search in global memory is a
// chain of L2 round trips.
constexpr int kListSeq = 1024, kListTile = 2048;
__global__ void __launch_bounds__(1024) k_chunk_plan(ChunkArgs a, Plan p) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // k_chunk_attn may set itself up
  __shared__ int64_t sh[32];
  __shared__ int64_t carry;
  __shared__ int32_t l_seq[kListSeq + 1];
  __shared__ int64_t l_cum[kListTile + 1];
  const int tid = threadIdx.x, nthr = blockDim.x;
  const csa2_cache &c = a.c;
  int32_t *seq_tile = c.batch <= kListSeq ? l_seq : p.seq_tile;
  // (needed two barriers further on)
  if (tid < c.batch && tid % 16 == 0) asm volatile("prefetch.global.L1 [%0];\n" ::"l"(c.n_tokens + tid));
  if (tid == 0) {
    carry = 0;
    seq_tile[0] = 0;
  }
  // where the list decreases, sequences may have rows in common
  int falls = 0;
  for (int b = tid; b < c.batch; b += nthr) falls |= a.cu[b + 1] < a.cu[b];
  falls = __syncthreads_or(falls);
  for (int b0 = 0; b0 < c.batch; b0 += nthr) {  // row tiles of each sequence
    const int b = b0 + tid;
    int first = 0, n = 0;
    if (b < c.batch && !ragged_rows(a.cu, b, a.total, a.max_new, first, n)) raise_err(a.err, CSA2_DEVERR_INDEX);
    if (falls && n > 0 && !ragged_own(a.cu, c.batch, b, first, n)) n = 0;
    const int64_t rt = (static_cast<int64_t>(n) * a.heads + kRows - 1) / kRows;
    const int64_t incl = block_scan(rt, sh) + carry;
    if (b < c.batch) seq_tile[b + 1] = static_cast<int32_t>(min(incl, static_cast<int64_t>(p.max_tiles)));
    __syncthreads();
    if (tid == nthr - 1) carry = incl;
    __syncthreads();
  }
  const int n_tiles = static_cast<int>(min(carry, static_cast<int64_t>(p.max_tiles)));
  const bool fits = n_tiles <= kListTile;
  int64_t *cum = fits ? l_cum : p.cum;
  __syncthreads();
  if (tid == 0) {
    carry = 0;
    cum[0] = 0;
    p.cum[0] = 0;
  }
  __syncthreads();
  for (int t0 = 0; t0 < n_tiles; t0 += nthr) {
    const int t = t0 + tid;
    int64_t units = 0;
    if (t < n_tiles) {
      const int b = last_at_most(seq_tile, c.batch, t);
      int first, n;
      ragged_rows(a.cu, b, a.total, a.max_new, first, n);
      const int64_t P = c.n_tokens[b] - n;
      const int64_t r0 = static_cast<int64_t>(t - seq_tile[b]) * kRows;  // within the sequence
      const int64_t left = static_cast<int64_t>(n) * a.heads - r0;
      // (rows of a call fit 31 bits: total is at most 2^24, heads 2^7)
      const uint32_t tok0 = static_cast<uint32_t>(r0) / static_cast<uint32_t>(a.heads);
      RowTile x{};
      x.seq = b;
      x.nrows = static_cast<int>(left < kRows ? left : kRows);
      x.row0 = static_cast<int64_t>(first) * a.heads + r0;
      x.head0 = static_cast<int>(r0 - static_cast<int64_t>(tok0) * a.heads);
      const uint32_t tok1 = tok0 + static_cast<uint32_t>(x.head0 + x.nrows - 1) / static_cast<uint32_t>(a.heads);
      x.pos0 = P + tok0;
      x.win0 = static_cast<int64_t>(first) + static_cast<int64_t>(kWin) * b + tok0 + 1;
      x.T = static_cast<int>(visible(P + tok1, c.ratio, c.capacity));
      x.nkeys = x.T + kWin + static_cast<int>(tok1 - tok0);
      x.ntiles = (x.nkeys + kKeys - 1) / kKeys;
      p.tile[t] = x;
      units = x.ntiles + 1;
    }
    const int64_t incl = block_scan(units, sh) + carry;
    if (t < n_tiles) {
      p.cum[t + 1] = incl;
      if (fits) cum[t + 1] = incl;
    }
    __syncthreads();
    if (tid == nthr - 1) carry = incl;
    __syncthreads();
  }
  const int64_t W = carry;
  __shared__ int32_t n_merge;
  if (tid == 0) n_merge = 0;
  __syncthreads();
  // no more CTAs than units (one token over 1,000 entries takes 25.7 us with a unit
  // each, 26.6 with two)
  const int64_t g_eff = max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.n_cta), W));
  for (int g = tid; g < p.n_cta; g += nthr) {
    CtaRange r{};
    if (g < g_eff && W > 0) {
      r.lo = W * g / g_eff;
      r.hi = W * (g + 1) / g_eff;
      r.tile = last_at_most<int64_t>(cum, n_tiles, r.lo);
      const int64_t c0 = cum[r.tile], nt = cum[r.tile + 1] - c0 - 1;
      if (r.lo > c0 && r.lo < c0 + nt && r.hi >= c0 + nt) {
        int first = static_cast<int>(c0 * g_eff / W);  // the CTA of unit c0, give or take a rounding
        while (first > 0 && W * first / g_eff > c0) --first;
        while (W * (first + 1) / g_eff <= c0) ++first;
        // (in any order: each joins rows of its own)
        p.merge[atomicAdd(&n_merge, 1)] = make_int4(g, first, r.tile, 0);
      }
    }
    p.cta[g] = r;
  }
  __syncthreads();
  for (int i = n_merge + tid; i < p.n_cta; i += nthr) p.merge[i] = make_int4(-1, 0, 0, 0);
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
// Issued by one elected lane of a warp whose control flow is uniform: the
// descriptors then live in uniform registers and a step's issue takes about 33
// cycles (61 from inside a one-lane branch), as long as the step itself.
__device__ __forceinline__ void mma_f16(uint32_t elected, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (elected)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
// S[64 rows][64 keys] = Q K^T, K 16 per step
__device__ __forceinline__ void mma_qk(uint32_t elected, uint32_t d, uint64_t dq, uint64_t dk) {
  constexpr uint32_t id = (1u << 4) | ((kKeys >> 3) << 17) | ((kRows >> 4) << 24);
#pragma unroll
  for (int i = 0; i < 36; ++i)
    mma_f16(elected, d, dq + (((i / 4) * kBlk + 32 * (i % 4)) >> 4), dk + (((i / 4) * kBlk + 32 * (i % 4)) >> 4), id, i ? 1u : 0u);
}
// 128 dims of O^T[512 dims][64 rows] += V^T P^T, 16 keys per step; V^T MN-major
__device__ __forceinline__ void mma_pv(uint32_t elected, uint32_t d, uint64_t dv, uint64_t dp, uint32_t acc) {
  constexpr uint32_t id = (1u << 4) | (1u << 15) | ((kRows >> 3) << 17) | ((128u >> 4) << 24);
#pragma unroll
  for (int i = 0; i < 4; ++i) mma_f16(elected, d, dv + ((2048 * i) >> 4), dp + ((32 * i) >> 4), id, i ? 1u : acc);
}
__device__ __forceinline__ void tmem_st_x1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(v) : "memory");
}
// 16 lanes x 32 columns, the lanes' rows spread over the warp: thread t gets
// columns 8 j + 2 (t % 4) + {0, 1} of row t / 4 in r[4 j], r[4 j + 1] and of row
// t / 4 + 8 in r[4 j + 2], r[4 j + 3].  Waits.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
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

// One key tile of the CTA, as the ahead warp lists it for the producers.
struct TileRef {
  int64_t base;  // physical entry of its first key; -1: not 64 whole entries; kNoTile after the last one
  int32_t t, kt;
};
constexpr int64_t kNoTile = -2;
constexpr int kRing = 16;

struct __align__(1024) ChunkSmem {
  uint8_t k[2][kBlocks][kBlk];      // two key tiles in fp16; block 8 (RoPE) then holds the tile's P
  uint8_t q[kBlocks][kBlk];
  __align__(16) float alpha[kRows]; // rescale of a row's O^T column in this tile (1: none)
  __align__(16) float fin[kRows];   // output factor of the finished item's rows
  __align__(16) float2 sg[2][kKeys]; // sigma of each key (-inf: no key) and 2^sigma
  float f[kRows];                   // logit factor of each row
  uint32_t moved[2][2];             // rows whose reference moves in a tile (by its parity)
  float tmax[2][kRows], lsum[kRows];  // row maxima of a tile's halves; sums of the second half
  int32_t vis[kRows], w0[kRows];    // a row sees keys j < vis and w0 <= j < w0 + 128
  __align__(16) uint8_t plain[2][kPrWarps];  // a producer warp's keys are all valid with sigma 0
  uint32_t tmem, progress;          // progress: the key tile (of this CTA's) being filled
  uint32_t listed;                  // key tiles in the ring so far
  __align__(16) TileRef ring[kRing];
  __align__(8) uint64_t full[2];      // tile filled
  __align__(8) uint64_t empty[2];     // ... and its PV complete
  // by tile parity, both: S of tile n + 1 may be issued before P of tile n has been
  // waited for, so P of tile n + 1 may arrive before that wait, and a parity wait
  // cannot tell a phase from the one two further on
  __align__(8) uint64_t s_full[2], p_full[2];
  __align__(8) uint64_t q_ready;
};

// Whether a phase is complete, without waiting; the same answer in every lane.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(tc::smem_addr(bar)), "r"(parity)
      : "memory");
  return __any_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, int32_t *err) {
  const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(bar, parity, kWaitIters));
  if (!ok && (threadIdx.x & 31) == 0) raise_err(err, CSA2_DEVERR_TIMEOUT);
  return ok;
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

// The work items of one CTA, in order: key tiles [k0, k1) of row tile t.  (Kept
// small: what is needed once per item is read again.)
struct Items {
  int t, k0, k1;
  __device__ __forceinline__ Items(const Plan &p, int g) { t = p.cta[g].tile - 1; }
  __device__ __forceinline__ const RowTile *x(const Plan &p) const { return p.tile + t; }
  __device__ __forceinline__ bool next(const Plan &p, int g) {
    const int64_t lo = p.cta[g].lo, hi = p.cta[g].hi;
    if (hi <= lo) return false;
    for (;;) {
      const int64_t c0 = p.cum[++t];
      if (c0 >= hi || t >= p.max_tiles) return false;
      const int nt = p.tile[t].ntiles;
      k0 = static_cast<int>(lo > c0 ? lo - c0 : 0);
      k1 = static_cast<int>(hi - c0 < nt ? hi - c0 : nt);
      if (k0 < k1) return true;
    }
  }
};

// sigma of a key whose largest magnitude is about 2^e: zero while fp16 holds the
// values as they are, else what brings the largest to about 2^8.
__device__ __forceinline__ int sigma_of(int e) {
  if (e < -1000 || (e >= 0 && e <= 15)) return 0;
  return max(-24, min(120, e - 8));
}

// ------------------------------------------------------------------ filling a tile
// Eight neighbouring threads per key.  A step is one 16-byte load per thread, 128
// contiguous bytes of a key's record (the load unit looks up one line per eight
// lanes; with four keys' lines there instead the fill was 10 % slower): 256 FP4
// dims (two steps) or 128 FP8 dims (four), then the RoPE dims.  The records come
// through registers, requested a whole tile ahead (and into L2 further ahead, by
// the ahead warp).
struct RawFp4 {
  static constexpr bool kFp4 = true;
  static constexpr int kSteps = 3;
  uint4 w[2];
  uint32_t r, sc[5];  // a step's two scales; prepared: each as an fp16 pair
};
struct RawFp8 {
  static constexpr bool kFp4 = false;
  static constexpr int kSteps = 5;
  uint4 w[5];
  uint4 sc;  // the key's 16 scales: word s holds those of step s; prepared: the factor of step s
};
__device__ __forceinline__ void load_step(const csa2_cache &c, int64_t e, int o, int s, RawFp4 &r) {
  if (s < 2) {
    r.w[s] = ldg16(c.lat_codes + e * 256 + 128 * s + 16 * o);
    r.sc[2 * s] = __ldg(reinterpret_cast<const uint16_t *>(c.lat_scales + e * 32 + 16 * s + 2 * o));
  } else {
    r.r = __ldg(reinterpret_cast<const uint32_t *>(c.rope_codes + e * 32 + 4 * o));
    r.sc[4] = __ldg(c.rope_scales + e * 4 + (o >> 1));
  }
}
__device__ __forceinline__ void load_step(const csa2_cache &c, int64_t e, int o, int s, RawFp8 &r) {
  r.w[s] = ldg16(s < 4 ? c.lat_codes + e * 512 + 128 * s + 16 * o : c.rope_codes + e * 128 + 16 * o);
  if (s == 4) r.sc = ldg16(c.lat_scales + e * 16);
}

__device__ __forceinline__ uint4 dq_e2m1(uint32_t w, uint32_t s2) {
  uint32_t h[4];
  e2m1x8_h2(w, h);
  return make_uint4(hmul2u(h[0], s2), hmul2u(h[1], s2), hmul2u(h[2], s2), hmul2u(h[3], s2));
}
__device__ __forceinline__ uint4 dq_e4m3(uint32_t w0, uint32_t w1, uint32_t m2) {
  uint32_t h[4];
  e4m3x8_h2(w0, w1, h);
  return make_uint4(hmul2u(h[0], m2), hmul2u(h[1], m2), hmul2u(h[2], m2), hmul2u(h[3], m2));
}
// 16-byte chunk x (8 dims) of key (or query row) `key` in a 64-dim block
__device__ __forceinline__ uint8_t *chunk_at(uint8_t *blk, int key, int x) { return blk + key * 128 + ((x ^ (key & 7)) << 4); }
// The two chunks of a thread's 16 dims of step s: lo = its first 8 dims.  The
// threads of the second 64-dim block (o >= 4) store theirs in the other order, so
// that a key's eight threads hit eight different 16 B banks at a time.
__device__ __forceinline__ void put_step(uint8_t (*k)[kBlk], int s, int key, int o, uint4 lo, uint4 hi) {
  const int flip = o >> 2;
  uint8_t *blk = k[2 * s + flip];
  const int x = 2 * (o & 3);
  *reinterpret_cast<uint4 *>(chunk_at(blk, key, x + flip)) = flip ? hi : lo;
  *reinterpret_cast<uint4 *>(chunk_at(blk, key, x + (flip ^ 1))) = flip ? lo : hi;
}
__device__ __forceinline__ void swap_if(bool p, uint32_t &a, uint32_t &b) {
  const uint32_t t = p ? b : a;
  b = p ? a : b;
  a = t;
}
// What can be done with a key's registers before its buffer is free: the scales as
// factors, and the order of the chunks.  Of a step's four chunks thread o stores
// its chunk j ^ (o / 2) as the j-th, so that a key's eight threads hit eight
// different 16 B banks at a time.
__device__ __forceinline__ void prepare(RawFp4 &r, int o, int) {
  const bool p1 = o & 2, p2 = o & 4;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    swap_if(p1, r.w[s].x, r.w[s].y);
    swap_if(p1, r.w[s].z, r.w[s].w);
    swap_if(p2, r.w[s].x, r.w[s].z);
    swap_if(p2, r.w[s].y, r.w[s].w);
    const uint32_t two = r.sc[2 * s];
    r.sc[2 * s] = e4m3x2_h2(__byte_perm(two, 0, p2 ? 0x11 : 0x00));
    r.sc[2 * s + 1] = e4m3x2_h2(__byte_perm(two, 0, p2 ? 0x00 : 0x11));
  }
  r.sc[4] = e4m3x2_h2(__byte_perm(r.sc[4], 0, 0x00));
}
__device__ __forceinline__ void store_step(uint8_t (*k)[kBlk], int s, int key, int o, const RawFp4 &r) {
  if (s < 2) {
    uint8_t *blk = k[4 * s + (o >> 1)];
    const int x = 4 * (o & 1) + (o >> 1);
    *reinterpret_cast<uint4 *>(chunk_at(blk, key, x)) = dq_e2m1(r.w[s].x, r.sc[2 * s]);
    *reinterpret_cast<uint4 *>(chunk_at(blk, key, x ^ 1)) = dq_e2m1(r.w[s].y, r.sc[2 * s]);
    *reinterpret_cast<uint4 *>(chunk_at(blk, key, x ^ 2)) = dq_e2m1(r.w[s].z, r.sc[2 * s + 1]);
    *reinterpret_cast<uint4 *>(chunk_at(blk, key, x ^ 3)) = dq_e2m1(r.w[s].w, r.sc[2 * s + 1]);
  } else {
    *reinterpret_cast<uint4 *>(chunk_at(k[8], key, o)) = dq_e2m1(r.r, r.sc[4]);
  }
}
// factor 2^k as an fp16 pair (k <= 15; zero below fp16's least, 2^-24)
__device__ __forceinline__ uint32_t pow2_h2(int k) {
  const uint32_t h = k < -24 ? 0u : k < -14 ? 1u << (k + 24) : static_cast<uint32_t>(k + 15) << 10;
  return h * 0x10001u;
}
__device__ __forceinline__ uint4 bf16x8_h(uint4 v, float inv) {
  return make_uint4(pack_h2(__uint_as_float(v.x << 16) * inv, __uint_as_float(v.x & 0xFFFF0000u) * inv),
                    pack_h2(__uint_as_float(v.y << 16) * inv, __uint_as_float(v.y & 0xFFFF0000u) * inv),
                    pack_h2(__uint_as_float(v.z << 16) * inv, __uint_as_float(v.z & 0xFFFF0000u) * inv),
                    pack_h2(__uint_as_float(v.w << 16) * inv, __uint_as_float(v.w & 0xFFFF0000u) * inv));
}
// A block whose factor 2^k fp16 does not have: 2^k x = 2^-24 (2^(k+24) x), with
// 2^(k+24) x rounded to E4M3 codes again, which only its step of 2^-9 near zero can
// change: by 2^-34 at most, of values that fp16 then rounds to its step of 2^-24.
// Returns the factor's exponent that is left.
__device__ __forceinline__ int rescale_block(uint4 &w, int k) {
  if (k >= -24) return k;
  const uint32_t m2 = pow2_h2(k + 24);
  uint32_t *u[4] = {&w.x, &w.y, &w.z, &w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(lo) : "r"(hmul2u(e4m3x2_h2(*u[i] & 0xFFFF), m2)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(hi) : "r"(hmul2u(e4m3x2_h2(*u[i] >> 16), m2)));
    *u[i] = lo | (static_cast<uint32_t>(hi) << 16);
  }
  return -24;
}
__device__ __forceinline__ uint32_t word_of(uint4 v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// The scales of a thread's blocks, one per step.
__device__ __forceinline__ uint4 own_scales(const RawFp8 &r, int o) {
  const int shift = 8 * (o >> 1);
  return make_uint4((r.sc.x >> shift) & 0xFF, (r.sc.y >> shift) & 0xFF, (r.sc.z >> shift) & 0xFF, (r.sc.w >> shift) & 0xFF);
}
__device__ __forceinline__ void prepare(RawFp8 &r, int o, int sigma) {
  const int off = 127 + sigma;
  const uint4 k = own_scales(r, o);
  r.sc.x = pow2_h2(static_cast<int>(k.x) - off);
  r.sc.y = pow2_h2(static_cast<int>(k.y) - off);
  r.sc.z = pow2_h2(static_cast<int>(k.z) - off);
  r.sc.w = pow2_h2(static_cast<int>(k.w) - off);
  r.w[4] = bf16x8_h(r.w[4], pow2f(-sigma));  // 8 RoPE dims in bf16
}
__device__ __forceinline__ void store_step(uint8_t (*k)[kBlk], int s, int key, int o, const RawFp8 &r) {
  if (s < 4) {
    const uint32_t m2 = word_of(r.sc, s);
    put_step(k, s, key, o, dq_e4m3(r.w[s].x, r.w[s].y, m2), dq_e4m3(r.w[s].z, r.w[s].w, m2));
  } else {
    *reinterpret_cast<uint4 *>(chunk_at(k[8], key, o)) = r.w[4];
  }
}
__device__ __forceinline__ int e8m0_top(uint4 s) {  // largest of 16 scale bytes
  uint32_t m = __vmaxu4(__vmaxu4(s.x, s.y), __vmaxu4(s.z, s.w));
  m = __vmaxu4(m, m >> 16);
  return max(m & 0xFF, (m >> 8) & 0xFF);
}
__device__ __forceinline__ uint32_t bf16_top(uint4 v, uint32_t m) {  // largest magnitude bits of 8 bf16
  const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
  return __vmaxu2(m, __vmaxu2(a, b));
}
__device__ __forceinline__ uint32_t key_max(uint32_t bf) {  // over the eight threads of a key
  bf = __vmaxu2(bf, __shfl_xor_sync(0xffffffffu, bf, 1));
  bf = __vmaxu2(bf, __shfl_xor_sync(0xffffffffu, bf, 2));
  return __vmaxu2(bf, __shfl_xor_sync(0xffffffffu, bf, 4));
}
// exponent e (largest magnitude about 2^e) of a key: an E8M0 top (block maximum
// about 2^(top - 119)) and / or the largest bf16 magnitude
__device__ __forceinline__ int key_exponent(int e8, uint32_t bf) {
  const int mb = max(bf & 0xFFFF, bf >> 16);
  const int a = e8 > 0 ? e8 - 119 : -2000, b = mb > 0 ? (mb >> 7) - 127 : -2000;
  return max(a, b);
}
// Whether a thread's part of a record has blocks (not of zeros, scale 0) whose factor
// fp16 does not have: such a tile is filled by fill_tail, which has code for them.
// (The same code here as well, in a branch that is hardly ever taken: 1,024 queries over
// V4 entries 3.57 ms against 3.54.)
__device__ __forceinline__ bool small_blocks(const RawFp4 &, int, int) { return false; }
__device__ __forceinline__ bool small_blocks(const RawFp8 &r, int o, int sigma) {
  const uint4 k = own_scales(r, o);
  return min(min(k.x - 1u, k.y - 1u), min(k.z - 1u, k.w - 1u)) < static_cast<uint32_t>(127 + sigma - 24 - 1);
}
__device__ __forceinline__ int raw_sigma(const RawFp4 &, int) { return 0; }
__device__ __forceinline__ int raw_sigma(const RawFp8 &r, int o) {
  // (two threads of the key have the same scales)
  const uint4 k = own_scales(r, o);
  const uint32_t bf = bf16_top(r.w[4], 0);
  const uint32_t both = key_max(max(max(k.x, k.y), max(k.z, k.w)) | max(bf & 0xFFFF, bf >> 16) << 16);
  return sigma_of(key_exponent(static_cast<int>(both & 0xFFFF), both >> 16));
}

// A tile that is not made of whole entries alone: key j is entry j (j < T), a
// window token, or nothing.
struct TailKey {
  int kind;  // 0 nothing, 1 FP4 entry, 2 V4 entry, 3 MXFP8 window row, 4 bf16 window row
  const uint8_t *codes, *scales, *rope, *rope_scales;
};
__device__ __forceinline__ void tail_key(const ChunkArgs &a, const RowTile &x, int64_t j, TailKey &k) {
  const csa2_cache &c = a.c;
  k.kind = 0;
  if (j < x.T) {
    const int64_t e = entry_at(c, x.seq, static_cast<int>(j));
    if (e < 0) {
      raise_err(a.err, CSA2_DEVERR_INDEX);
      return;
    }
    const bool fp8 = c.entry_format == CSA2_ENTRY_FP8;
    k.kind = fp8 ? 2 : 1;
    k.codes = c.lat_codes + e * (fp8 ? 512 : 256);
    k.scales = c.lat_scales + e * (fp8 ? 16 : 32);
    k.rope = c.rope_codes + e * (fp8 ? 128 : 32);
    k.rope_scales = fp8 ? nullptr : c.rope_scales + e * 4;
  } else if (j < x.nkeys) {
    const int64_t tok = x.pos0 - (kWin - 1) + (j - x.T);
    if (tok < 0) return;
    const uint8_t *codes = c.swa_codes, *scales = c.swa_scales;
    int64_t at = static_cast<int64_t>(x.seq) * kWin + (tok & (kWin - 1));
    if (a.win_codes != nullptr) {
      codes = a.win_codes;
      scales = a.win_scales;
      at = x.win0 + (j - x.T);
    } else if (tok < c.n_tokens[x.seq] - kWin) {
      raise_err(a.err, CSA2_DEVERR_INDEX);
      return;
    }
    const bool fp8 = c.swa_dtype == CSA2_SWA_MXFP8;
    k.kind = fp8 ? 3 : 4;
    k.codes = codes + at * (fp8 ? 576 : 1152);
    k.scales = fp8 ? scales + at * kSwaScaleStride : nullptr;
    k.rope = k.codes + (fp8 ? 512 : 1024);
    k.rope_scales = fp8 ? k.scales + 16 : nullptr;
  }
}
struct RawTail {
  uint4 w[2];
  uint32_t sc;
};
__device__ __forceinline__ void tail_load(const TailKey &k, int s, int o, RawTail &r) {
  if (k.kind == 1) {
    if (s < 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(k.codes + 64 * s + 8 * o));
      r.w[0].x = v.x, r.w[0].y = v.y;
      r.sc = __ldg(k.scales + 8 * s + o);
    } else {
      r.w[0].x = __ldg(reinterpret_cast<const uint32_t *>(k.rope + 4 * o));
      r.sc = __ldg(k.rope_scales + (o >> 1));
    }
  } else if (k.kind == 3 && s == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(k.rope + 8 * o));
    r.w[0].x = v.x, r.w[0].y = v.y;
    r.sc = __ldg(k.rope_scales + (o >> 2));
  } else if (k.kind == 2 || k.kind == 3) {
    r.w[0] = ldg16(s < 4 ? k.codes + 128 * s + 16 * o : k.rope + 16 * o);
    if (s < 4) r.sc = __ldg(k.scales + 4 * s + (o >> 1));
  } else if (k.kind == 4) {
    const uint8_t *src = s < 4 ? k.codes + 256 * s + 32 * o : k.rope + 16 * o;
    r.w[0] = ldg16(src);
    if (s < 4) r.w[1] = ldg16(src + 16);
  }
}
__device__ __forceinline__ void tail_store(uint8_t (*k)[kBlk], const TailKey &t, int s, int key, int o, const RawTail &r, int sigma) {
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (t.kind == 1) {
    const uint32_t s2 = e4m3x2_h2(r.sc * 0x101);
    lo = dq_e2m1(r.w[0].x, s2);
    hi = dq_e2m1(r.w[0].y, s2);
  } else if (t.kind == 4 || (t.kind == 2 && s == 4)) {
    const float inv = pow2f(-sigma);
    lo = bf16x8_h(r.w[0], inv);
    hi = bf16x8_h(r.w[1], inv);
  } else if (t.kind) {
    uint4 w = r.w[0];
    const uint32_t m2 = pow2_h2(rescale_block(w, static_cast<int>(r.sc) - 127 - sigma));
    lo = dq_e4m3(w.x, w.y, m2);
    hi = dq_e4m3(w.z, w.w, m2);
  }
  if (s < 4) put_step(k, s, key, o, lo, hi);
  else *reinterpret_cast<uint4 *>(chunk_at(k[8], key, o)) = lo;
}

// Physical entry of the first key of key tile kt, or -1 when the tile is not 64
// whole entries of one valid page.
__device__ __forceinline__ int64_t whole_tile(const csa2_cache &c, int seq, int T, int kt) {
  if ((kt + 1) * static_cast<int64_t>(kKeys) > T) return -1;
  return entry_at(c, seq, kt * kKeys);
}

// All of a thread's part is requested at once, before the wait for the buffer.
__device__ __noinline__ bool fill_tail(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, uint32_t n, int pt, bool dead) {
  const int key = pt >> 3, o = pt & 7, b = n & 1;
  TailKey t;
  tail_key(a, p.tile[sm.ring[n % kRing].t], static_cast<int64_t>(sm.ring[n % kRing].kt) * kKeys + key, t);
  RawTail r[5];
#pragma unroll
  for (int s = 0; s < 5; ++s) tail_load(t, s, o, r[s]);
  int e8 = 0;
  uint32_t bf = 0, lat = 0;  // largest magnitude bits of all bf16 values, of a bf16 window's latents
  if (t.kind == 2) {
    e8 = e8m0_top(ldg16(t.scales));
    bf = bf16_top(r[4].w[0], 0);
  } else if (t.kind == 3) {
    e8 = max(e8m0_top(ldg16(t.scales)), static_cast<int>(max(__ldg(t.rope_scales), __ldg(t.rope_scales + 1))));
  } else if (t.kind == 4) {
#pragma unroll
    for (int s = 0; s < 4; ++s) lat = bf16_top(r[s].w[1], bf16_top(r[s].w[0], lat));
    bf = bf16_top(r[4].w[0], lat);
  }
  bf = key_max(bf);
  lat = key_max(lat);
  // A latent that is infinite or NaN would reach every row of the tile in PV (0 x it),
  // also those that do not see the key.  The key's latents go in as zeros, and its
  // logit is NaN for the rows that do.
  const bool poison = max(lat & 0xFFFF, lat >> 16) >= 0x7F80;
  if (poison) {
#pragma unroll
    for (int s = 0; s < 4; ++s) r[s].w[0] = r[s].w[1] = make_uint4(0, 0, 0, 0);
  }
  const int sigma = t.kind >= 2 ? sigma_of(key_exponent(e8, bf)) : 0;
  if (n >= 2 && !dead) dead = !wait_warp(&sm.empty[b], ((n >> 1) & 1) ^ 1, a.err);
  if (pt == 0) *const_cast<volatile uint32_t *>(&sm.progress) = n;
  if ((pt & 31) == 0) sm.plain[b][pt >> 5] = 0;
  if (o == 0)
    sm.sg[b][key] = t.kind ? make_float2(poison ? NAN : static_cast<float>(sigma), pow2f(sigma)) : make_float2(-INFINITY, 0.0f);
#pragma unroll
  for (int s = 0; s < 5; ++s) tail_store(sm.k[b], t, s, key, o, r[s], sigma);
  return dead;
}

// The producer warps: tile n into buffer n % 2 once the PV that read it last is
// complete.  Which tiles, and where they lie, they are told through the ring:
// a page-table load of their own would wait behind the records' loads.
__device__ __forceinline__ int64_t ring_base(const ChunkSmem &sm, uint32_t n, int32_t *err) {
  const volatile uint32_t *listed = &sm.listed;
  uint32_t i = 0;
  while (*listed <= n && i < kPolls) ++i;
  // (one answer for the warp: what follows has warp-wide operations)
  if (!__all_sync(0xffffffffu, *listed > n)) {
    if ((threadIdx.x & 31) == 0) raise_err(err, CSA2_DEVERR_TIMEOUT);
    return kNoTile;
  }
  __threadfence_block();
  return *const_cast<const volatile int64_t *>(&sm.ring[n % kRing].base);
}
template <class Raw>
__device__ __forceinline__ void produce(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, int pt) {
  const csa2_cache &c = a.c;
  const int key = pt >> 3, o = pt & 7;
  bool dead = false;
  Raw raw;
  int64_t base = ring_base(sm, 0, a.err);
  if (base >= 0) {
#pragma unroll
    for (int s = 0; s < Raw::kSteps; ++s) load_step(c, base + key, o, s, raw);
  }
  for (uint32_t n = 0; base != kNoTile; ++n) {
    const int b = n & 1;
    bool whole = base >= 0;
    base = ring_base(sm, n + 1, a.err);
    const int sigma = whole ? raw_sigma(raw, o) : 0;
    if (!Raw::kFp4) whole = whole && !__any_sync(0xffffffffu, small_blocks(raw, o, sigma));
    if (whole) {
      const bool plain = Raw::kFp4 || __all_sync(0xffffffffu, sigma == 0);
      prepare(raw, o, sigma);
      if (n >= 2 && !dead) dead = !wait_warp(&sm.empty[b], ((n >> 1) & 1) ^ 1, a.err);
      if (pt == 0) *const_cast<volatile uint32_t *>(&sm.progress) = n;
      if ((pt & 31) == 0) sm.plain[b][pt >> 5] = plain;
      if (o == 0) sm.sg[b][key] = make_float2(static_cast<float>(sigma), pow2f(sigma));
#pragma unroll
      for (int s = 0; s < Raw::kSteps; ++s) {
        store_step(sm.k[b], s, key, o, raw);
      }
    } else {
      dead = fill_tail(a, p, sm, n, pt, dead);
      raw = Raw{};
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if ((pt & 31) == 0) tc::mbar_arrive(&sm.full[b]);
    // (after the hand-over: the fence would wait for these loads too)
    if (base >= 0) {
#pragma unroll
      for (int s = 0; s < Raw::kSteps; ++s) load_step(c, base + key, o, s, raw);
    }
  }
}

// ------------------------------------------------------------------ query, softmax, read-out
// Query rows of an item to fp16 with a power-of-two scale per row, each row's
// logit factor and bounds.  Eight rows per warp.
__device__ __noinline__ void load_query(const ChunkArgs &a, const RowTile &x, ChunkSmem &sm, int warp, int lane) {
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
        sm.f[r] = pow2f(ex) * a.sm_scale * kLog2e;
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

// O^T of a finished item out of tensor memory: normalised rows, or (part) this
// CTA's part of a shared row tile.  Each warp has 32 dims of two blocks.
__device__ __noinline__ void read_out(const ChunkArgs &a, const ChunkSmem &sm, float *part, int64_t row0, int nrows,
                                      uint32_t tmem, int warp, int lane) {
  const int dim = 32 * (warp & 3) + lane;
  const uint32_t ta = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kColO;
#pragma unroll 1
  for (int i16 = 8 * (warp >> 2); i16 < 8 * (warp >> 2) + 8; ++i16) {
    const int b = i16 >> 2, h0 = 16 * (i16 & 3);
    uint32_t r[16];
    tc::tmem_ld_32x32b_x16(ta + 16 * i16, r);
    tc::tmem_ld_wait_x16(r);
    if (part != nullptr) {
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint4 *>(part + ((b * 16 + (h0 + i) / 4) * 128 + dim) * 4) =
            make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
    } else if (a.bf16) {
      // lane pairs exchange so that each stores two neighbouring dims of one row
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float v0 = __uint_as_float(r[i]) * sm.fin[h0 + i], v1 = __uint_as_float(r[i + 1]) * sm.fin[h0 + i + 1];
        const float o = __shfl_xor_sync(0xffffffffu, lane & 1 ? v0 : v1, 1);
        const int row = h0 + i + (lane & 1);
        const __nv_bfloat162 t2 = lane & 1 ? __floats2bfloat162_rn(o, v1) : __floats2bfloat162_rn(v0, o);
        if (row < nrows)
          *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + (row0 + row) * kLat + 128 * b +
                                              (dim & ~1)) = t2;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (h0 + i < nrows)
          static_cast<float *>(a.out)[(row0 + h0 + i) * kLat + 128 * b + dim] = __uint_as_float(r[i]) * sm.fin[h0 + i];
    }
  }
}

// The softmax warps: warps w and w + 4 have rows 16 w .. + 15 of S (TMEM lanes
// 32 w ..) and half of the keys each, a thread eight keys of rows ra and rb.  A
// row's reference maximum moves only when a weight would exceed 2^15 (fp16);
// the two warps then agree on it, and the row's O^T column is rescaled.
__device__ __forceinline__ void softmax(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, uint32_t tmem, int warp, int lane) {
  const int half = warp >> 2;
  const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const int ra = 16 * (warp & 3) + (lane >> 2), rb = ra + 8, col = 32 * half + 2 * (lane & 3);
  Items it(p, blockIdx.x);
  bool more = it.next(p, blockIdx.x), dead = false;
  uint32_t n = 0;  // tiles so far
  if (more) load_query(a, *it.x(p), sm, warp, lane);
  bar_softmax();
  while (more) {
    const RowTile *x = it.x(p);
    const int k0 = it.k0, k1 = it.k1;
    const float fa = sm.f[ra], fb = sm.f[rb];
    const int va = sm.vis[ra], vb = sm.vis[rb], wa = sm.w0[ra], wb = sm.w0[rb];
    float ma = 0.0f, mb = 0.0f, la = 0.0f, lb = 0.0f;  // reference (log2 units), this half's sum
    bool seen_a = false, seen_b = false;               // the reference is set
    for (int kt = k0; kt < k1; ++kt, ++n) {
      const int b = n & 1;
      if (!dead) dead = !wait_warp(&sm.full[b], (n >> 1) & 1, a.err);  // sg, plain of this tile
      if (!dead) dead = !wait_warp(&sm.s_full[b], (n >> 1) & 1, a.err);
      tc::tc_fence_after();
      float s[16];
      tmem_ld_rows16(tmem + lane_base + kColS + 64 * b + 32 * half, reinterpret_cast<uint32_t *>(s));
      // exponents of the weighted weights, x = z + sigma - m, and their row maxima
      float ta = -INFINITY, tb = -INFINITY;
      const uint4 pl = *reinterpret_cast<const uint4 *>(sm.plain[b]);
      const bool fast = (pl.x & pl.y & pl.z & pl.w) == 0x01010101u && (kt + 1) * kKeys <= va;  // (rb sees no less)
      if (fast) {
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          s[j] = fmaf(s[j], fa, -ma);
          s[j + 1] = fmaf(s[j + 1], fa, -ma);
          s[j + 2] = fmaf(s[j + 2], fb, -mb);
          s[j + 3] = fmaf(s[j + 3], fb, -mb);
          ta = fmaxf(ta, fmaxf(s[j], s[j + 1]));
          tb = fmaxf(tb, fmaxf(s[j + 2], s[j + 3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int k = 2 * j + col, key = kt * kKeys + k;
          const float4 g = *reinterpret_cast<const float4 *>(&sm.sg[b][k]);  // (sigma, 2^sigma) of two keys
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int kk = key + i;
            const float sg = i ? g.z : g.x, g2 = i ? g.w : g.y;
            const bool see_a = kk < va || (kk >= wa && kk < wa + kWin), see_b = kk < vb || (kk >= wb && kk < wb + kWin);
            s[j + i] = see_a ? fmaf(s[j + i] * g2, fa, sg - ma) : -INFINITY;
            s[j + 2 + i] = see_b ? fmaf(s[j + 2 + i] * g2, fb, sg - mb) : -INFINITY;
            ta = fmaxf(ta, s[j + i]);
            tb = fmaxf(tb, s[j + 2 + i]);
          }
        }
      }
      ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, 1));
      tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, 1));
      ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, 2));
      tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, 2));
      if ((lane & 3) == 0) {
        sm.tmax[half][ra] = ta;
        sm.tmax[half][rb] = tb;
      }
      const bool moving = bar_softmax_or(ta > (seen_a ? kSlack : -INFINITY) || tb > (seen_b ? kSlack : -INFINITY));
      // the next tile's list starts empty (the last tile's, in its place, has been read)
      if (warp == 0 && lane < 2) sm.moved[b ^ 1][lane] = 0;
      if (moving) {
        // some row's reference moves: both halves' maxima, the same decision in both
        ta = fmaxf(ta, sm.tmax[half ^ 1][ra]);
        tb = fmaxf(tb, sm.tmax[half ^ 1][rb]);
        const bool mva = ta > (seen_a ? kSlack : -INFINITY), mvb = tb > (seen_b ? kSlack : -INFINITY);
        const float da = mva ? ta - kTop : 0.0f, db = mvb ? tb - kTop : 0.0f;
        const float ala = mva ? (seen_a ? ex2(-da) : 0.0f) : 1.0f, alb = mvb ? (seen_b ? ex2(-db) : 0.0f) : 1.0f;
        ma += da;
        mb += db;
        la *= ala;
        lb *= alb;
        seen_a |= mva;
        seen_b |= mvb;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          s[j] -= da;
          s[j + 1] -= da;
          s[j + 2] -= db;
          s[j + 3] -= db;
        }
        if (half == 0 && (lane & 3) == 0) {
          if (mva) {
            sm.alpha[ra] = ala;
            atomicOr(&sm.moved[b][ra >> 5], 1u << (ra & 31));
          }
          if (mvb) {
            sm.alpha[rb] = alb;
            atomicOr(&sm.moved[b][rb >> 5], 1u << (rb & 31));
          }
        }
      }
      // weights: l in fp32 (without sigma), P to fp16 (with it; at most 2^15)
      uint8_t *pa = sm.k[b][8] + ra * 128 + 4 * (lane & 3), *pb = pa + 8 * 128;  // ra % 8 == rb % 8
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p0 = ex2(s[4 * j]), p1 = ex2(s[4 * j + 1]), p2 = ex2(s[4 * j + 2]), p3 = ex2(s[4 * j + 3]);
        if (fast) {
          la += p0 + p1;
          lb += p2 + p3;
        } else {
          const float4 g = *reinterpret_cast<const float4 *>(&sm.sg[b][8 * j + col]);
          const float g0 = ex2(-fmaxf(g.x, -126.0f)), g1 = ex2(-fmaxf(g.z, -126.0f));
          la = fmaf(p0, g0, fmaf(p1, g1, la));
          lb = fmaf(p2, g0, fmaf(p3, g1, lb));
        }
        const int at = ((4 * half + j) ^ (ra & 7)) << 4;
        *reinterpret_cast<uint32_t *>(pa + at) = pack_h2(p0, p1);
        *reinterpret_cast<uint32_t *>(pb + at) = pack_h2(p2, p3);
      }
      if (moving) {
        // the moved rows' O^T columns follow, once the last PV is complete (this
        // comes after the weights: they do not depend on it)
        bar_softmax();
        uint32_t todo = sm.moved[b][half];  // this warp's share: rows 32 half .., its 32 dims of each block
        if (kt > k0) {
          if (!dead) dead = !wait_warp(&sm.empty[b ^ 1], ((n - 1) >> 1) & 1, a.err);
          tc::tc_fence_after();
          const uint32_t at = tmem + lane_base + kColO + 32 * half;
          while (todo) {  // four rows' columns of the four blocks in flight together
            int row[4];
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              row[i] = todo ? __ffs(todo) - 1 : row[0];
              todo &= todo - 1;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) tc::tmem_ld_32x32b_x1(at + 64 * (i & 3) + row[i >> 2], r[i]);
            tc::tmem_ld_wait_x16(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float v = __uint_as_float(r[i]) * sm.alpha[32 * half + row[i >> 2]];
              tmem_st_x1(at + 64 * (i & 3) + row[i >> 2], __float_as_uint(v));
            }
          }
          asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
        }
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.p_full[b]);
    }
    // ---- the item's last PV is on its way: sums, output factors, the next query
    la += __shfl_xor_sync(0xffffffffu, la, 1);
    lb += __shfl_xor_sync(0xffffffffu, lb, 1);
    la += __shfl_xor_sync(0xffffffffu, la, 2);
    lb += __shfl_xor_sync(0xffffffffu, lb, 2);
    if (half == 1 && (lane & 3) == 0) {
      sm.lsum[ra] = la;
      sm.lsum[rb] = lb;
    }
    bar_softmax();
    const bool direct = k0 == 0 && k1 == x->ntiles;
    float *part = direct ? nullptr : p.part + (2 * blockIdx.x + (k0 > 0 ? 0 : 1)) * kPartFloats;
    if (half == 0 && (lane & 3) < 2) {  // lane 0 of a row's four: ra, lane 1: rb
      const bool second = lane & 1;
      const int r = second ? rb : ra;
      float m = second ? (seen_b ? mb : -INFINITY) : (seen_a ? ma : -INFINITY), sum = (second ? lb : la) + sm.lsum[r];
      if (!direct) {
        *reinterpret_cast<float2 *>(part + kLat * kRows + 2 * r) = make_float2(m, sum);
      } else {
        float f = 1.0f;
        if (a.sink != nullptr) {
          const float z = a.sink[(x->head0 + r) % a.heads] * kLog2e;
          const float mf = fmaxf(m, z);
          f = m == -INFINITY ? 0.0f : ex2(m - mf);
          sum = sum * f + (z == mf ? 1.0f : ex2(z - mf));  // (an infinite sink too)
          m = mf;
        }
        // (0: a row without keys; NaN stays NaN)
        sm.fin[r] = sum == 0.0f ? 0.0f : f / sum;
        if (r < x->nrows && !dead) a.lse[x->row0 + r] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
      }
    }
    more = it.next(p, blockIdx.x);
    if (more) load_query(a, *it.x(p), sm, warp, lane);  // (S of the last tile is complete)
    bar_softmax();                                      // fin, the next rows' data
    if (!dead) dead = !wait_warp(&sm.empty[(n - 1) & 1], ((n - 1) >> 1) & 1, a.err);
    tc::tc_fence_after();
    if (!dead) read_out(a, sm, part, x->row0, x->nrows, tmem, warp, lane);
    tc::tc_fence_before();
    // (fin is written again only after another item's barriers)
  }
}

// ------------------------------------------------------------------ MMA issuer
// Per key tile: S = Q K^T once the tile is filled, PV once its P is there.  The
// S of the next tile is issued before the PV of this one whenever that tile is
// ready first, so that the tensor cores work while the softmax does.
__device__ __forceinline__ void issue(const ChunkArgs &a, const Plan &p, ChunkSmem &sm, uint32_t tmem) {
  const uint32_t e = elect_one();
  const uint32_t ka = tc::smem_addr(sm.k);
  const uint64_t dq = desc_sw128(tc::smem_addr(sm.q), 16, 1024), dk = desc_sw128(ka, 16, 1024);
  const uint64_t dv = desc_sw128(ka, kBlk, 1024), dp = desc_sw128(ka + 8 * kBlk, 16, 1024);
  Items it(p, blockIdx.x);
  uint32_t n = 0, items = 0;
  auto qk = [&](uint32_t t) {
    tc::tc_fence_after();
    mma_qk(e, tmem + kColS + 64 * (t & 1), dq, dk + (t & 1) * (kTile >> 4));
    if (e) tc::mma_commit(&sm.s_full[t & 1]);
  };
  while (it.next(p, blockIdx.x)) {
    const int tiles = it.k1 - it.k0;
    if (!wait_warp(&sm.q_ready, items & 1, a.err)) return;
    ++items;
    bool ahead = false;  // S of tile n is issued
    for (int i = 0; i < tiles; ++i, ++n) {
      if (!ahead) {
        if (!wait_warp(&sm.full[n & 1], (n >> 1) & 1, a.err)) return;
        qk(n);
      }
      ahead = false;
      // whichever comes first: the next tile, or this one's P (bounded polls that
      // do not suspend while either may come)
      bool ready = false;
      for (uint32_t poll = 0; !ready && !ahead && i + 1 < tiles && poll < kPolls; ++poll) {
        ready = mbar_test(&sm.p_full[n & 1], (n >> 1) & 1);
        if (!ready && mbar_test(&sm.full[(n + 1) & 1], ((n + 1) >> 1) & 1)) {
          ahead = true;
          qk(n + 1);
        }
      }
      if (!ready && !wait_warp(&sm.p_full[n & 1], (n >> 1) & 1, a.err)) return;
      tc::tc_fence_after();
      const uint32_t buf = (n & 1) * (kTile >> 4);
#pragma unroll 1
      for (int blk = 0; blk < 4; ++blk)
        mma_pv(e, tmem + kColO + 64 * blk, dv + buf + ((2 * kBlk * blk) >> 4), dp + buf, i > 0 ? 1u : 0u);
      if (e) tc::mma_commit(&sm.empty[n & 1]);
    }
  }
}

// One thread that lists the CTA's coming key tiles for the producers and asks
// for their records: whole tiles are contiguous in every plane, so a few bulk
// prefetches into L2 each.
__device__ __forceinline__ void prefetch_l2(const uint8_t *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ahead(const ChunkArgs &a, const Plan &p, ChunkSmem &sm) {
  const csa2_cache &c = a.c;
  const volatile uint32_t *progress = &sm.progress;
  Items it(p, blockIdx.x);
  uint32_t n = 0;
  auto list = [&](int64_t base, int t, int kt) {
    volatile TileRef *r = &sm.ring[n % kRing];
    r->base = base;
    r->t = t;
    r->kt = kt;
    __threadfence_block();
    *const_cast<volatile uint32_t *>(&sm.listed) = ++n;
  };
  while (it.next(p, blockIdx.x)) {
    const int seq = it.x(p)->seq, T = it.x(p)->T;
    for (int kt = it.k0; kt < it.k1; ++kt) {
      const int64_t base = whole_tile(c, seq, T, kt);
      // not further ahead than the ring and the L2 should hold (bounded: a stopped
      // producer has raised its own error)
      uint32_t i = 0;
      while (*progress + kAhead < n && i < kPolls) {
        __nanosleep(100);
        ++i;
      }
      if (*progress + kAhead < n) {
        raise_err(a.err, CSA2_DEVERR_TIMEOUT);
        list(kNoTile, 0, 0);
        return;
      }
      list(base, it.t, kt);
      if (base < 0) continue;
      if (c.entry_format == CSA2_ENTRY_FP8) {
        prefetch_l2(c.lat_codes + base * 512, kKeys * 512);
        prefetch_l2(c.lat_scales + base * 16, kKeys * 16);
        prefetch_l2(c.rope_codes + base * 128, kKeys * 128);
      } else {
        prefetch_l2(c.lat_codes + base * 256, kKeys * 256);
        prefetch_l2(c.lat_scales + base * 32, kKeys * 32);
        prefetch_l2(c.rope_codes + base * 32, kKeys * 32);
        // (4 B per entry: in a dense cache the tile may start between two 16 B
        // boundaries, and a bulk prefetch may not)
        const uintptr_t rs = reinterpret_cast<uintptr_t>(c.rope_scales + base * 4);
        const uintptr_t r0 = (rs + 15) & ~uintptr_t(15), r1 = (rs + kKeys * 4) & ~uintptr_t(15);
        prefetch_l2(reinterpret_cast<const uint8_t *>(r0), static_cast<uint32_t>(r1 - r0));
      }
    }
  }
  list(kNoTile, 0, 0);
}

// One persistent CTA per SM: 8 softmax warps, 16 producer warps, the MMA warp, the
// ahead warp.  The work is dealt out in units of a key tile, so a decode batch of
// any shape fills the SMs; the parts of a shared row tile go through L2.
__global__ void __launch_bounds__(kThreads, 1) k_chunk_attn(const __grid_constant__ ChunkArgs a,
                                                             const __grid_constant__ Plan p) {
  // aligned by its declaration, not by arithmetic on the pointer, after which every
  // access would be a generic one with a 64-bit address
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem &sm = *reinterpret_cast<ChunkSmem *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.full[i], kPrWarps);
      tc::mbar_init(&sm.empty[i], 1);
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.p_full[i], kSmWarps);
    }
    tc::mbar_init(&sm.q_ready, kSmWarps);
    tc::fence_mbar_init();
    sm.progress = 0;
    sm.listed = 0;
    sm.moved[0][0] = sm.moved[0][1] = sm.moved[1][0] = sm.moved[1][1] = 0;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the plan is written
  if (warp < kSmWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kWorkRegs));
    softmax(a, p, sm, tmem, warp, lane);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kWorkRegs));
    if (a.c.entry_format == CSA2_ENTRY_FP8) produce<RawFp8>(a, p, sm, tid - 32 * kSmWarps);
    else produce<RawFp4>(a, p, sm, tid - 32 * kSmWarps);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kIssueRegs));
    if (warp == kMmaWarp) issue(a, p, sm, tmem);
    else if (warp == kAheadWarp && lane == 0) ahead(a, p, sm);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Row tiles shared by several CTAs: block (x, y) joins 8 rows x 128 kDims dims of
// the x-th of them, its parts in CTA order (part k is CTA first + k's).  A thread
// has kDims dims of four rows.  The parts lie in L2, so what counts is how many
// loads are in flight: eight per thread at once, the first of them before their
// weights are known, and with few row tiles (many parts each) four times the
// blocks.
constexpr int kMaxCta = 256;
template <int kDims>
__global__ void __launch_bounds__(256) k_chunk_merge(ChunkArgs a, Plan p) {
  constexpr int kSplit = 4 / kDims, kParts = 8 / kDims;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  __shared__ __align__(16) float wt[kMaxCta][8];  // (read four rows at a time)
  __shared__ float ls[kMaxCta][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int y = blockIdx.y / kSplit, b0 = blockIdx.y % kSplit * kDims;
  const int4 mg = p.merge[blockIdx.x];
  if (mg.x < 0) return;
  const int first = mg.y, n = mg.x - first + 1;
  // the first part is the last item of its CTA (slot 1), the others the first of theirs (slot 0)
  const float *part0 = p.part + (2 * first + 1) * kPartFloats, *part1 = p.part + 2 * (first + 1) * kPartFloats;
  auto part = [&](int k) { return k == 0 ? part0 : part1 + 2 * static_cast<int64_t>(k - 1) * kPartFloats; };
  const int d = threadIdx.x & 127, half = threadIdx.x >> 7, i4 = 2 * y + half;
  const int at4 = ((b0 * 16 + i4) * 128 + d) * 4;
  float4 v[kParts][kDims];
  auto load = [&](int k0) {
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (k0 + k < n) {
#pragma unroll
        for (int b = 0; b < kDims; ++b) v[k][b] = *reinterpret_cast<const float4 *>(part(k0 + k) + at4 + b * 16 * 128 * 4);
      }
  };
  load(0);
  const RowTile &x = p.tile[mg.z];
  const int nrows = x.nrows;
  if (8 * y >= nrows) return;
  const int64_t row0 = x.row0;
  {  // warp = row: the parts' weights, normalised
    const int r = 8 * y + warp;
    float m = -INFINITY, l = 0.0f;
    for (int k = lane; k < n; k += 32) {
      const float2 ml = *reinterpret_cast<const float2 *>(part(k) + kLat * kRows + 2 * r);
      wt[k][warp] = ml.x;
      ls[k][warp] = ml.y;
      m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int k = lane; k < n; k += 32) {  // (what this lane stored)
      const float mk = wt[k][warp], w = mk == -INFINITY ? 0.0f : ex2(mk - m);
      wt[k][warp] = w;
      l = fmaf(w, ls[k][warp], l);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float f = 1.0f;
    if (a.sink != nullptr) {
      const float z = a.sink[(x.head0 + r) % a.heads] * kLog2e, mf = fmaxf(m, z);
      f = m == -INFINITY ? 0.0f : ex2(m - mf);
      l = l * f + (z == mf ? 1.0f : ex2(z - mf));
      m = mf;
    }
    f = l == 0.0f ? 0.0f : f / l;
    for (int k = lane; k < n; k += 32) wt[k][warp] *= f;
    if (b0 == 0 && lane == 0 && r < nrows) a.lse[row0 + r] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
  __syncthreads();
  float o[kDims][4] = {};
  for (int k0 = 0;; k0 += kParts) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      if (k0 + k >= n) break;
      const float4 w = *reinterpret_cast<const float4 *>(&wt[k0 + k][4 * half]);
#pragma unroll
      for (int b = 0; b < kDims; ++b) {  // (a part without keys of a row holds nothing for it)
        o[b][0] = w.x == 0.0f ? o[b][0] : fmaf(w.x, v[k][b].x, o[b][0]);
        o[b][1] = w.y == 0.0f ? o[b][1] : fmaf(w.y, v[k][b].y, o[b][1]);
        o[b][2] = w.z == 0.0f ? o[b][2] : fmaf(w.z, v[k][b].z, o[b][2]);
        o[b][3] = w.w == 0.0f ? o[b][3] : fmaf(w.w, v[k][b].w, o[b][3]);
      }
    }
    if (k0 + kParts >= n) break;
    load(k0 + kParts);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * i4 + r;
    if (row >= nrows) break;
#pragma unroll
    for (int b = 0; b < kDims; ++b) {
      const int64_t at = (row0 + row) * kLat + 128 * (b0 + b) + d;
      if (a.bf16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(o[b][r]);
      else static_cast<float *>(a.out)[at] = o[b][r];
    }
  }
}

struct PlanLayout {
  size_t seq_tile, cum, tile, cta, merge, part, total;
  int max_tiles, n_cta;
};
PlanLayout plan_layout(int batch, int total, int heads) {
  PlanLayout L{};
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  const int64_t t = static_cast<int64_t>(total) * heads / kRows + (batch < total ? batch : total) + 1;
  L.max_tiles = static_cast<int>(t);
  L.n_cta = device_sm_count() < kMaxCta ? device_sm_count() : kMaxCta;
  size_t o = 0;
  L.seq_tile = o;
  o = up(o + (static_cast<size_t>(batch) + 1) * 4);
  L.cum = o;
  o = up(o + (static_cast<size_t>(t) + 1) * 8);
  L.tile = o;
  o = up(o + static_cast<size_t>(t) * sizeof(RowTile));
  L.cta = o;
  o = up(o + static_cast<size_t>(L.n_cta) * sizeof(CtaRange));
  L.merge = o;
  o = up(o + static_cast<size_t>(L.n_cta) * sizeof(int4));
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
               reinterpret_cast<int4 *>(wb + L.merge), reinterpret_cast<float *>(wb + L.part), L.max_tiles, L.n_cta};
  const int smem = static_cast<int>(sizeof(csa2::ChunkSmem)) + 1024;
  static_assert(sizeof(csa2::ChunkSmem) + 1024 <= 232448, "shared memory of one CTA");
  cudaError_t e = csa2::ensure_smem_limit(reinterpret_cast<const void *>(&csa2::k_chunk_attn), smem);
  if (e != cudaSuccess) return cuda_status(e, "csa2_chunk_attn shared memory");
  // (built with fewer registers at the launch, it would wait for some that do not exist)
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes at{};
    e = cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(&csa2::k_chunk_attn));
    if (e != cudaSuccess) return cuda_status(e, "csa2_chunk_attn attributes");
    regs.store(at.numRegs, std::memory_order_relaxed);
  }
  CSA2_REQUIRE(regs.load(std::memory_order_relaxed) >= csa2::kLaunchRegs, CSA2_ERR_CUDA,
               "csa2_chunk_attn was built with %d registers per thread", regs.load(std::memory_order_relaxed));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // (with 256 threads the barriers cost 2 us less: one token over 1,000 entries 23.7 us
  // against 25.7; more sequences or row tiles take passes, which 1,024 halve or better)
  csa2::k_chunk_plan<<<1, cache->batch <= 256 && L.max_tiles <= 256 ? 256 : 1024, 0, s>>>(a, p);
  e = cudaGetLastError();
  // each of the next two may set itself up while the one before still runs
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(L.n_cta);
    cfg.blockDim = dim3(csa2::kThreads);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, csa2::k_chunk_attn, a, p);
  }
  if (e == cudaSuccess) {
    // up to 64 shared row tiles: a block per 128 dims (over 152 CTAs, 4 row tiles take
    // 9.3 us against 12.5, 16 take 9.5 against 12.6, one of 40 parts 6.0 against 8.5);
    // more of them, of fewer parts each, fill the SMs without (65: 9.2 us against
    // 10.6; 152: 12.7 against 24.0)
    const int shared = L.n_cta < L.max_tiles ? L.n_cta : L.max_tiles, split = shared <= 64 ? 4 : 1;
    cfg.gridDim = dim3(shared, csa2::kRows / 8 * split);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = split == 4 ? cudaLaunchKernelEx(&cfg, csa2::k_chunk_merge<1>, a, p)
                   : cudaLaunchKernelEx(&cfg, csa2::k_chunk_merge<4>, a, p);
  }
  return cuda_status(e, "csa2_chunk_attn launch");
}

}  // extern "C"
