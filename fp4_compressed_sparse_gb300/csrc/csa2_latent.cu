// csa2_latent.cu -- the two products that lead into the latent space and out of it
// ([P2] "DeepSeek Multi-Head Latent Attention(MLA) 해부" §4: the key's and the value's
// up-projections absorbed into the query and the output), per head h:
//   csa2_query_latent   q[t, h, 0:512]   = sum_k q_nope[t, h, k] W_UK[h, k, 0:512]
//                       q[t, h, 512:576] = RoPE(q_rope[t, h], pos[t])
//   csa2_value_project  o[t, h, j]       = sum_c o_latent[t, h, c] W_UV[h, j, c]
// on the tcgen05 tensor cores in bf16, sums in fp32 in tensor memory.
//
// Work and bound.  2 x 512 x dim flop per (token, head) against 2 (dim + 64) + 1152
// bytes (query) or 1024 + 2 dim (value, bf16): 90 and 100 flop per byte at dim 128, a
// third of what the tensor cores need to be the bound.  HBM bounds long batches, the
// chain of loads short ones.
//
// Two forms, by the number of tokens (both sides' times stand at few_queries): a block per
// head and column part with everything in flight at once (csa2_latent_few.cu), and the
// persistent kernel of this file.  fp32 latents are cut into three bf16 parts that add up to
// them, each multiplied: the sums are of the values as they were given.
//
// Measured (in a graph, caches as the calls before leave them): 4,001 tokens of 64 heads of
// 128: queries 73 us (403 MB, 5.5 TB/s, 81 % of the measured copy rate), values bf16 56 us
// (336 MB, 6.0 TB/s, 88 %), fp32 104 us (599 MB, 5.8 TB/s); 128 tokens: 5.8, 4.4 and 8.4 us
// (fp32: a chain of 16 stages, each cut into its parts).  Tensor pipe 18, 22 and 39 %.  Short of
// the copy rate: the reload of W when a CTA's run passes to another head (nothing is computed
// meanwhile), rows of 1,152 B at 74 KB distance out.
#include "csa2_latent.cuh"
#include "csa2_tc.cuh"
#include "csa2_tma.cuh"

namespace csa2 {
namespace {

constexpr int kTok = 128;                   // tokens of a tile
constexpr uint32_t kWaitIters = 200;        // suspended polls of <= 1 ms each
constexpr int kWBytes = 128 * kLat * 2;     // 128 KB: a head's W, or a part of it
constexpr int kBox = kTok * 128;            // 128 rows of 128 bytes, 128-byte swizzle
enum Mode { kQuery, kValue, kValueF32 };

// Beside W: stages of the tokens' rows, and for queries what is on its way out.  A stage is
// what one wait and arming of the copying thread (0.2 us) is worth: 32 KB, two boxes of 64
// columns (query: all of a tile's; value: a quarter), fp32: one of 32.
template <Mode kM>
struct Shape {
  static constexpr int kStage = kM == kValueF32 ? kBox : 2 * kBox;
  static constexpr int kStages = kM == kValueF32 ? 6 : kM == kQuery ? 2 : 3;
  static constexpr int kOut = kM == kQuery ? 8 * 4096 : 0;  // 4 KB per writing warp
  static constexpr int kBytes = kWBytes + kStages * kStage + kOut + 1024;
  static constexpr int kMoreWarps = kM == kValue ? 0 : 8;  // that rotate, or split
  static constexpr int kThreads = 32 * (12 + kMoreWarps);
};
// fp32 latents: their bf16 parts lie in tensor memory, as the MMA's rows, 16 columns of a
// buffer each, behind two accumulators of 128 columns: one for the first parts, one for the
// others, 2^-8 as large.  An MMA's sums lose what lies below fp32's last bit, so in one accumulator
// the two small parts' steps cost as much as the first's: of 8 million values 1.1 in 1,000 were
// not the rounded 64-bit ones, so it is 0.27 (a plain fp32 product: 0.29).  The sums are read out
// between two units, which takes 2.5 % (4,001 tokens 104.5 us; 102 with one for all parts, double).
constexpr int kPartBufs = 4, kRestCol = 128, kPartCol = 256, kPartCols = 64;
struct Sync {
  uint64_t full[6], empty[6];
  uint64_t wfull[4], wdone;      // W, or a stage's columns of it, has landed; the last MMAs that read it are done
  uint64_t pfull[kPartBufs], pempty[kPartBufs];  // fp32: the bf16 parts
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  uint32_t loaded, w_loaded;     // stages armed, and copies of W
  int dead;                      // a wait gave up
};

__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t phase) {
  return __all_sync(0xffffffffu, tc::mbar_wait_bounded(bar, phase, kWaitIters));
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
__device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
               "l"(map), "r"(c0), "r"(c1), "r"(tc::smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
               "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_addr(bar))
               : "memory");
}
// kind::f16, bf16 x bf16 -> fp32, M 128
__device__ __forceinline__ uint32_t idesc_bf16(int n, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kTok >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with its rows in tensor memory (a lane each, two values a column).
__device__ __forceinline__ void mma_bf16_rows(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 128-byte swizzle.  K-major: sbo between 8-row groups.  MN-major (64 values of N per
// row, a row per k): lbo between 64-value blocks along N, sbo between groups of 8 k.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFF) >> 4) | static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts4(uint32_t at, const uint32_t *v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// 16 bf16 values; wide: dst is on a boundary of 32 bytes.
__device__ __forceinline__ void put16(uint16_t *dst, const uint32_t *o, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]),
                 "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// One persistent CTA per SM.  A unit is (head, column part, tile of 128 tokens), done in one
// job or, queries with all of their 512 columns, in two of 256; units of a head and part
// follow one another and a CTA takes a run of jobs, so that its part of W stays in shared
// memory.  Tokens are the MMA's 128 rows (a lane holds one token and
// writes runs of its row), W's columns its N.
//   warp 0       copies W (once per head and part) and the tokens' rows, by tensor maps
//   warp 1       issues the MMAs
//   warps 4-11   read the sums out of tensor memory and write them: two groups of four,
//                one per accumulator (fp32 latents: both on every unit)
//   warps 12-    query: rotate the RoPE dims, from global memory to global memory;
//                fp32 latents: cut a stage into three bf16 parts in tensor memory
template <Mode kM>
__global__ void __launch_bounds__(Shape<kM>::kThreads, 1)
    k_latent(LatentArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
             const __grid_constant__ CUtensorMap mo) {
  using S = Shape<kM>;
  constexpr bool kQ = kM == kQuery, kF = kM == kValueF32;
  // bf16 values: W comes in four groups of 128 columns, each just before the stage that is multiplied
  // by it (1,000 tokens of 64 heads 13.4 us against 14.7 with all of W first; for the others that
  // gained nothing)
  constexpr int kWGroups = kM == kValue ? 4 : 1;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(128) Sync sy;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t s_w = (tc::smem_addr(raw) + 1023) & ~1023u, s_x = s_w + kWBytes, s_p = s_x + S::kStages * S::kStage;
  const int jobs = kQ && a.np > 256 ? 2 : 1, cols = a.np / jobs;  // accumulators of a unit, their columns
  const int chunks = kQ ? 1 : kF ? kLat / 32 : kLat / 128;       // stages of a unit
  // this CTA's jobs: job v is of unit v >> shift (up to 2^27 jobs); whole units unless a.halves
  const int shift = jobs - 1, keep = a.halves ? 0 : shift;
  const int64_t shares = static_cast<int64_t>(a.heads) * a.parts * a.tiles << (shift - keep);
  const int v0 = static_cast<int>(shares * blockIdx.x / gridDim.x) << keep;
  const int v1 = static_cast<int>(shares * (blockIdx.x + 1) / gridDim.x) << keep;
  if (warp == 1) {
    tc::tmem_alloc(&sy.tmem, 512);
    tc::tmem_relinquish();
  }
  if (t == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      tc::mbar_init(&sy.full[i], 1);
      tc::mbar_init(&sy.empty[i], kF ? 4 : 1);
    }
    for (int i = 0; i < kPartBufs; ++i) {
      tc::mbar_init(&sy.pfull[i], 4);
      tc::mbar_init(&sy.pempty[i], 1);
    }
    for (int i = 0; i < kWGroups; ++i) tc::mbar_init(&sy.wfull[i], 1);
    tc::mbar_init(&sy.wdone, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sy.tfull[i], 1);
      tc::mbar_init(&sy.tempty[i], kF ? 8 : 4);
    }
    sy.loaded = sy.w_loaded = 0;
    sy.dead = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  next_may_start();
  wait_for_previous();
  const uint32_t tmem = sy.tmem;
  auto gave_up = [&]() {
    raise_err(a.err, CSA2_DEVERR_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sy.dead) = 1;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    const uint32_t el = elect_one();
    const int boxes = kQ ? (a.dim + 63) / 64 : kF ? 1 : 2, wide = kF ? 32 : 64;
    const int w_boxes = kQ ? a.np / 64 : kLat / 64, w_box = (kQ ? a.dim : a.np) * 128;
    int held = -1;
    uint32_t n = 0, st = 0, ph = 1, wn = 0;  // wn: copies of W so far
    bool ok = true;
    for (int u = v0 >> shift; u << shift < v1 && ok; ++u) {
      const int hp = u / a.tiles, tile = u - hp * a.tiles, h = hp / a.parts, part = hp - h * a.parts;
      auto w_group = [&](int g, int n_box) {
        if (el) {
          tc::mbar_expect_tx(&sy.wfull[g], n_box * w_box);
          for (int i = g * n_box; i < (g + 1) * n_box; ++i)
            load3(s_w + i * w_box, &mw, (kQ ? part * a.np : 0) + 64 * i, kQ ? 0 : part * a.np, h, &sy.wfull[g]);
        }
        __syncwarp();
      };
      if (hp != held) {
        if (wn > 0) ok = wait_all(&sy.wdone, (wn - 1) & 1);
        if (!ok) break;
        ++wn;
        if (kWGroups == 1) w_group(0, w_boxes);
      }
      const bool fresh = hp != held;
      held = hp;
      for (int c = 0; c < chunks; ++c, ++n) {
        if (kWGroups > 1 && fresh) w_group(c, 2);
        if (n >= S::kStages) ok = wait_all(&sy.empty[st], ph);
        if (!ok) break;
        if (el) {
          tc::mbar_expect_tx(&sy.full[st], boxes * kBox);
          for (int i = 0; i < boxes; ++i)
            load2(s_x + st * S::kStage + i * kBox, &mx, (kQ ? h * (a.dim + kRope) : h * kLat + c * (kF ? 32 : 128)) + wide * i, tile * kTok, &sy.full[st]);
        }
        __syncwarp();
        if (++st == S::kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (lane == 0) {
      sy.loaded = n;
      sy.w_loaded = wn;
      if (!ok) gave_up();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    const uint32_t el = elect_one(), id = idesc_bf16(cols, kQ ? 1 : 0);
    int held = -1;
    uint32_t st = 0, ph = 0, j = 0, wn = 0;
    bool ok = true;
    for (int v = v0; v < v1 && ok; ++v, ++j) {
      const int hp = (v >> shift) / a.tiles, b = v & shift;
      const bool first = b == 0 || v == v0, last = b == jobs - 1 || v == v1 - 1;  // of the unit's jobs here
      const bool fresh = hp != held;
      if (fresh) {
        if (kWGroups == 1) ok = wait_all(&sy.wfull[0], wn & 1);
        ++wn;
        held = hp;
      }
      if (ok) {
        const uint32_t acc = kF ? 0 : j & 1, d = tmem + 256 * acc;
        if (kF && j >= 1) ok = wait_all(&sy.tempty[0], (j - 1) & 1);
        if (!kF && j >= 2) ok = wait_all(&sy.tempty[acc], ((j >> 1) - 1) & 1);
        for (int c = 0; c < chunks && ok; ++c) {
          if (kWGroups > 1 && fresh) ok = wait_all(&sy.wfull[c], (wn - 1) & 1);
          if (first && ok) ok = kF ? wait_all(&sy.pfull[st], ph) : wait_all(&sy.full[st], ph);
          if (!ok) break;
          tc::tc_fence_after();
          if (el) {
            if constexpr (kQ) {
              const uint64_t dx = desc_sw128(s_x + st * S::kStage, 16, 1024);
              const uint64_t dw = desc_sw128(s_w + b * (cols / 64) * a.dim * 128, a.dim * 128, 1024);
              for (int s = 0; s < a.dim / 16; ++s)
                mma_bf16(d, dx + (((s >> 2) * kBox + 32 * (s & 3)) >> 4), dw + (2048 * s >> 4), id, s > 0 ? 1u : 0u);
            } else if constexpr (kF) {
              const uint64_t dw = desc_sw128(s_w + (c >> 1) * a.np * 128, 16, 1024) + (64 * (c & 1) >> 4);
              const uint32_t tx = tmem + kPartCol + kPartCols * st;
#pragma unroll
              for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int z = 0; z < 3; ++z)
                  mma_bf16_rows(z == 0 ? d : d + kRestCol, tx + 16 * z + 8 * s, dw + (32 * s >> 4), id, c + s > 0 || z == 2 ? 1u : 0u);
            } else {
              const uint64_t dx = desc_sw128(s_x + st * S::kStage, 16, 1024);
#pragma unroll
              for (int s = 0; s < 8; ++s)
                mma_bf16(d, dx + (((s >> 2) * kBox + 32 * (s & 3)) >> 4),
                         desc_sw128(s_w + (2 * c + (s >> 2)) * a.np * 128, 16, 1024) + (32 * (s & 3) >> 4), id, c + s > 0 ? 1u : 0u);
            }
            if (last) tc::mma_commit(kF ? &sy.pempty[st] : &sy.empty[st]);
            if (c == chunks - 1) {
              tc::mma_commit(&sy.tfull[acc]);
              if (v + 1 < v1 && (v + 1 >> shift) / a.tiles != hp) tc::mma_commit(&sy.wdone);
            }
          }
          __syncwarp();
          if (last && ++st == (kF ? kPartBufs : S::kStages)) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
    if (!ok && lane == 0) gave_up();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ results
    const int q = warp & 3, g = (warp - 4) >> 2;
    uint32_t j = 0;
    bool ok = true;
    for (int v = v0; v < v1 && ok; ++v, ++j) {
      const int u = v >> shift, b = v & shift, hp = u / a.tiles, tile = u - hp * a.tiles, h = hp / a.parts, part = hp - h * a.parts;
      const int64_t tok = static_cast<int64_t>(tile) * kTok + 32 * q + lane;
      if constexpr (kF) {  // both groups, every second 16 columns each; the sums are free before the stores
        ok = wait_all(&sy.tfull[0], j & 1);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + 16 * g;
        uint32_t o[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (16 * g + 32 * i >= cols) break;
          uint32_t r[16], rest[16];
          tc::tmem_ld_32x32b_x16(at + 32 * i, r);
          tc::tmem_ld_32x32b_x16(at + kRestCol + 32 * i, rest);
          tc::tmem_ld_wait_x16(r);
          tc::tmem_ld_wait_x16(rest);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[i][k] = pack_bf16(__uint_as_float(r[2 * k]) + __uint_as_float(rest[2 * k]), __uint_as_float(r[2 * k + 1]) + __uint_as_float(rest[2 * k + 1]));
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sy.tempty[0]);
        uint16_t *dst = a.out + tok * a.out_stride + static_cast<int64_t>(h) * a.dim + part * a.np + 16 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tok < a.total && 16 * g + 32 * i < cols) put16(dst + 32 * i, o[i], a.wide);
      } else if ((j & 1) == g) {
        bool live = tok < a.total;
        int64_t p;
        if (kQ && live) live = row_position(a, tok, false, p);
        uint16_t *dst = a.out + tok * a.out_stride + (kQ ? static_cast<int64_t>(h) * kDqk : static_cast<int64_t>(h) * a.dim) +
                        part * a.np + b * cols;
        ok = wait_all(&sy.tfull[g], (j >> 1) & 1);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t at = tmem + 256 * g + (static_cast<uint32_t>(32 * q) << 16);
        // Whole rows of queries go out as boxes of 32 tokens x 64 columns through shared
        // memory (a lane's own 32-byte stores of 1,152-byte rows take 1.3 times as long).
        if (kQ && __all_sync(0xffffffffu, live || tok >= a.total)) {
          const uint32_t buf = s_p + (warp - 4) * 4096;
          for (int c = 0; c < cols; c += 64) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t r[16], o[8];
              tc::tmem_ld_32x32b_x16(at + c + 16 * i, r);
              tc::tmem_ld_wait_x16(r);
#pragma unroll
              for (int v = 0; v < 8; ++v) o[v] = pack_bf16(__uint_as_float(r[2 * v]), __uint_as_float(r[2 * v + 1]));
              sts4(buf + lane * 128 + (((2 * i) ^ (lane & 7)) << 4), o);
              sts4(buf + lane * 128 + (((2 * i + 1) ^ (lane & 7)) << 4), o + 4);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(&mo),
                           "r"(h * kDqk + part * a.np + b * cols + c), "r"(tile * kTok + 32 * q), "r"(buf)
                           : "memory");
              asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
            }
          }
        } else {
          for (int c = 0; c < cols; c += 16) {
            uint32_t r[16], o[8];
            tc::tmem_ld_32x32b_x16(at + c, r);
            tc::tmem_ld_wait_x16(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
            if (live) put16(dst + c, o, a.wide);
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sy.tempty[g]);
      }
    }
    if (!ok && lane == 0) gave_up();
  } else if (kQ && warp >= 12) {
    // ------------------------------------------------------------ RoPE: a lane takes 8 dims of four tokens
    // (all of a unit's loads at once, the positions a unit ahead: a chain of two loads
    // per unit took longer than its bytes)
    const int d8 = lane & 7, r0 = 4 * (warp - 12) + (lane >> 3);
    const int u0 = (v0 + shift) >> shift, u1 = (v1 + shift) >> shift;  // units whose first job is here
    int64_t p[4];
    auto positions = [&](int u) {
      const int hp = u / a.tiles;
      const int64_t t0 = static_cast<int64_t>(u - hp * a.tiles) * kTok;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t tok = t0 + r0 + 32 * i;
        if (u >= u1 || tok >= a.total || !row_position(a, tok, hp == 0 && d8 == 0, p[i])) p[i] = -1;
      }
    };
    positions(u0);
    for (int u = u0; u < u1; ++u) {
      const int hp = u / a.tiles, h = hp / a.parts;
      const int64_t t0 = static_cast<int64_t>(u - hp * a.tiles) * kTok;
      const bool mine = hp % a.parts == 0;
      const uint16_t *src = static_cast<const uint16_t *>(a.x) + (t0 + r0) * a.x_stride + h * (a.dim + kRope) + a.dim + 8 * d8;
      Rope8 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (mine && p[i] >= 0) x[i] = load_rope8(a, src + 32 * i * a.x_stride, p[i], d8);
      bool there[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) there[i] = mine && p[i] >= 0;
      positions(u + 1);
      uint16_t *dst = a.out + (t0 + r0) * a.out_stride + h * kDqk + kLat + 8 * d8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (there[i]) store_rope8(x[i], dst + 32 * i * a.out_stride);
    }
  } else if (kF && warp >= 12) {
    // ------------------------------------------------------------ fp32 stages to bf16 parts
    // (two groups of four warps, each every second stage: while one waits the other splits; a
    // lane takes a token's 32 values)
    const int r8 = lane & 7;
    const uint32_t n_all = static_cast<uint32_t>(v1 - v0) * chunks, quarter = 32 * (warp & 3);
    bool ok = true;
    for (uint32_t n = (warp - 12) >> 2; n < n_all; n += 2) {
      const uint32_t st = n % S::kStages, pb = n % kPartBufs, use = n / kPartBufs;
      ok = wait_all(&sy.full[st], (n / S::kStages) & 1) && (use == 0 || wait_all(&sy.pempty[pb], (use - 1) & 1));
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t src = s_x + st * S::kStage + (quarter + lane) * 128, dst = tmem + (quarter << 16) + kPartCol + kPartCols * pb;
      uint32_t part[3][16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = lds4(src + ((i ^ r8) << 4));
        uint32_t p[2][3];
        split3(v.x, v.y, p[0]);
        split3(v.z, v.w, p[1]);
#pragma unroll
        for (int z = 0; z < 3; ++z) part[z][2 * i] = p[0][z], part[z][2 * i + 1] = p[1][z];
      }
#pragma unroll
      for (int z = 0; z < 3; ++z) tmem_st_x16(dst + 16 * z, part[z]);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sy.empty[st]);
      asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sy.pfull[pb]);
    }
    if (!ok && lane == 0) gave_up();
  }
  if (kQ && warp >= 4 && warp < 12 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  tc::tc_fence_before();
  __syncthreads();
  if (t == 0 && sy.dead) {  // copies still in flight
    for (uint32_t i = sy.loaded > S::kStages ? sy.loaded - S::kStages : 0; i < sy.loaded; ++i)
      tc::mbar_wait_bounded(&sy.full[i % S::kStages], (i / S::kStages) & 1, kWaitIters);
    for (int i = 0; i < kWGroups && sy.w_loaded > 0; ++i) tc::mbar_wait_bounded(&sy.wfull[i], (sy.w_loaded - 1) & 1, kWaitIters);
  }
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <Mode kM>
cudaError_t launch(const LatentArgs &a, cudaStream_t s) {
  const auto kern = k_latent<kM>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), Shape<kM>::kBytes);
  if (e != cudaSuccess) return e;
  constexpr bool kQ = kM == kQuery, kF = kM == kValueF32;
  CUtensorMap mx, mw, mo{};
  const uint64_t elt = kF ? 4 : 2;
  const uint64_t x_dim[2] = {static_cast<uint64_t>(a.heads) * (kQ ? a.dim + kRope : kLat), static_cast<uint64_t>(a.total)};
  const uint64_t x_stride[1] = {static_cast<uint64_t>(a.x_stride) * elt};
  const uint32_t x_box[2] = {kF ? 32u : 64u, kTok};
  const uint64_t w_dim[3] = {kLat, static_cast<uint64_t>(a.dim), static_cast<uint64_t>(a.heads)};
  const uint64_t w_stride[2] = {kLat * 2, static_cast<uint64_t>(a.w_stride) * 2};
  const uint32_t w_box[3] = {64, static_cast<uint32_t>(kQ ? a.dim : a.np), 1};
  if (!tensor_map(&mx, kF ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.x, x_dim, x_stride, x_box, true) ||
      !tensor_map(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.w, w_dim, w_stride, w_box, true))
    return cudaErrorNotSupported;
  if constexpr (kQ) {
    const uint64_t o_dim[2] = {static_cast<uint64_t>(a.out_stride), static_cast<uint64_t>(a.total)}, o_stride[1] = {a.out_stride * 2ull};
    const uint32_t o_box[2] = {64, 32};
    if (!tensor_map(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, o_dim, o_stride, o_box, true)) return cudaErrorNotSupported;
  }
  const int64_t shares = static_cast<int64_t>(a.heads) * a.parts * a.tiles << a.halves, sms = device_sm_count();
  return launch_after(kern, dim3(static_cast<unsigned>(shares < sms ? shares : sms)), Shape<kM>::kThreads, Shape<kM>::kBytes, 0, s, a, mx, mw, mo);
}

}  // namespace
}  // namespace csa2

extern "C" {

using csa2::cuda_status;

csa2_status csa2_query_latent(const uint16_t *q, int64_t q_stride, int32_t total, int32_t n_heads, int32_t dim,
                              const uint16_t *w_uk, int64_t w_stride, const int64_t *pos, const float *rope_cs,
                              int64_t rope_len, uint16_t *out, int32_t *err_word, csa2_stream_t stream) {
  CSA2_REQUIRE(total >= 0 && total <= (1 << 24), CSA2_ERR_SHAPE, "total %d outside 0..2^24", total);
  CSA2_REQUIRE(n_heads >= 1 && n_heads <= CSA2_MAX_HEADS, CSA2_ERR_SHAPE, "n_heads %d outside 1..128", n_heads);
  CSA2_REQUIRE(dim >= 16 && dim <= 128 && dim % 16 == 0, CSA2_ERR_SHAPE, "dim %d must be a multiple of 16, 16..128", dim);
  CSA2_REQUIRE_PTR(w_uk);
  CSA2_REQUIRE_PTR(rope_cs);
  CSA2_REQUIRE(rope_len >= 1, CSA2_ERR_SHAPE, "rope_len %lld < 1", static_cast<long long>(rope_len));
  CSA2_REQUIRE(q_stride >= static_cast<int64_t>(n_heads) * (dim + CSA2_D_ROPE) && q_stride % 8 == 0, CSA2_ERR_SHAPE,
               "q_stride %lld must be a multiple of 8, n_heads x (dim + 64) at least", static_cast<long long>(q_stride));
  CSA2_REQUIRE(w_stride >= static_cast<int64_t>(dim) * CSA2_D_LATENT && w_stride % 8 == 0, CSA2_ERR_SHAPE,
               "w_stride %lld must be a multiple of 8, dim x 512 at least", static_cast<long long>(w_stride));
  if (total == 0) return CSA2_OK;
  CSA2_REQUIRE_PTR(q);
  CSA2_REQUIRE_PTR(pos);
  CSA2_REQUIRE_PTR(out);
  csa2::LatentArgs a{};
  a.x = q;
  a.x_stride = q_stride;
  a.w = w_uk;
  a.w_stride = w_stride;
  a.heads = n_heads;
  a.dim = dim;
  a.total = total;
  a.pos = pos;
  a.rope = rope_cs;
  a.rope_len = rope_len;
  a.out = out;
  a.out_stride = static_cast<int64_t>(n_heads) * CSA2_D_QK;
  a.tiles = (total + csa2::kTok - 1) / csa2::kTok;
  a.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  a.err = err_word;
  if (csa2::few_queries(total, n_heads))
    return cuda_status(csa2::launch_query_few(a, reinterpret_cast<cudaStream_t>(stream)), "csa2_query_latent launch");
  // A CTA for every SM: columns in parts while heads and tiles are too few for that.  Else runs
  // of whole units, or, where that makes the longest run shorter, of halves: in two parts up to
  // two units per CTA (384 tokens of 64 heads 9.6 us against 10.3 by halves and 11.2), by a run's
  // ends above (1,000 tokens 20.7 against 22.5); where it does not, 250 tokens 8.2 against 7.0.
  const int64_t units = static_cast<int64_t>(n_heads) * a.tiles, sms = csa2::device_sm_count();
  const bool shorter = (2 * units + sms - 1) / sms < 2 * ((units + sms - 1) / sms);
  a.parts = 4 * units <= sms ? 4 : 2 * units <= sms || (shorter && units <= 2 * sms) ? 2 : 1;
  a.halves = a.parts == 1 && shorter;
  a.np = CSA2_D_LATENT / a.parts;
  return cuda_status(csa2::launch<csa2::kQuery>(a, reinterpret_cast<cudaStream_t>(stream)), "csa2_query_latent launch");
}

csa2_status csa2_value_project(const void *o, int64_t o_stride, int32_t in_dtype, int32_t total, int32_t n_heads, int32_t dim,
                               const uint16_t *w_uv, int64_t w_stride, uint16_t *out, int64_t out_stride, int32_t *err_word,
                               csa2_stream_t stream) {
  CSA2_REQUIRE(total >= 0 && total <= (1 << 24), CSA2_ERR_SHAPE, "total %d outside 0..2^24", total);
  CSA2_REQUIRE(n_heads >= 1 && n_heads <= CSA2_MAX_HEADS, CSA2_ERR_SHAPE, "n_heads %d outside 1..128", n_heads);
  CSA2_REQUIRE(dim >= 16 && dim <= 128 && dim % 16 == 0, CSA2_ERR_SHAPE, "dim %d must be a multiple of 16, 16..128", dim);
  CSA2_REQUIRE(in_dtype == CSA2_IN_F32 || in_dtype == CSA2_IN_BF16, CSA2_ERR_RANGE, "in_dtype %d", in_dtype);
  CSA2_REQUIRE_PTR(w_uv);
  CSA2_REQUIRE(o_stride >= static_cast<int64_t>(n_heads) * CSA2_D_LATENT && o_stride % 8 == 0, CSA2_ERR_SHAPE,
               "o_stride %lld must be a multiple of 8, n_heads x 512 at least", static_cast<long long>(o_stride));
  CSA2_REQUIRE(w_stride >= static_cast<int64_t>(dim) * CSA2_D_LATENT && w_stride % 8 == 0, CSA2_ERR_SHAPE,
               "w_stride %lld must be a multiple of 8, dim x 512 at least", static_cast<long long>(w_stride));
  CSA2_REQUIRE(out_stride >= static_cast<int64_t>(n_heads) * dim && out_stride % 8 == 0, CSA2_ERR_SHAPE,
               "out_stride %lld must be a multiple of 8, n_heads x dim at least", static_cast<long long>(out_stride));
  if (total == 0) return CSA2_OK;
  CSA2_REQUIRE_PTR(o);
  CSA2_REQUIRE_PTR(out);
  csa2::LatentArgs a{};
  a.x = o;
  a.x_stride = o_stride;
  a.w = w_uv;
  a.w_stride = w_stride;
  a.heads = n_heads;
  a.dim = dim;
  a.total = total;
  a.out = out;
  a.out_stride = out_stride;
  a.tiles = (total + csa2::kTok - 1) / csa2::kTok;
  a.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && out_stride % 16 == 0;
  a.err = err_word;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (csa2::few_values(total, n_heads, dim, in_dtype == CSA2_IN_F32))
    return cuda_status(csa2::launch_value_few(a, in_dtype == CSA2_IN_F32, s), "csa2_value_project launch");
  const int64_t units = static_cast<int64_t>(n_heads) * a.tiles, sms = csa2::device_sm_count();
  a.parts = 1;
  while (2 * units * a.parts <= sms && dim % (32 * a.parts) == 0 && a.parts < 4) a.parts *= 2;
  a.np = dim / a.parts;
  return cuda_status(in_dtype == CSA2_IN_F32 ? csa2::launch<csa2::kValueF32>(a, s) : csa2::launch<csa2::kValue>(a, s),
                     "csa2_value_project launch");
}

}  // extern "C"
