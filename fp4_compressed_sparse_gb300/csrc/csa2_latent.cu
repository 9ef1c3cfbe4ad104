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
// Three forms, by the number of tokens and the latents' type (the launch rules have both
// sides' times):
//   k_query_few, k_value_few   a block per head and column part, W from global memory
//                              straight into the fragments of mma.sync: one round of loads
//   k_latent                   persistent, tcgen05, operands by tensor maps
//   k_value_f32                the same for fp32 latents, which warps split into bf16 parts
//                              hi + lo, each multiplied: what is lost is 2^-16 of a value,
//                              against 2^-8 that the bf16 result's rounding takes
#include "csa2_latent.cuh"
#include "csa2_tc.cuh"

namespace csa2 {
namespace {

constexpr int kTok = 128;                       // tokens of a tile
constexpr int kLoadWarps = 8, kOutWarps = 8;
constexpr int kThreads = 32 * (kLoadWarps + kOutWarps + 1);
constexpr int kIssueWarp = kLoadWarps + kOutWarps;
constexpr uint32_t kWaitIters = 200;
constexpr int kWBytesMax = 128 * kLat * 2;      // 128 KB
constexpr int kMaxStages = 5;

struct Sync {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t wfull;
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
};

__device__ __forceinline__ bool wait1(uint64_t *bar, uint32_t phase, int32_t *err) {
  if (tc::mbar_wait_bounded(bar, phase, kWaitIters)) return true;
  raise_err(err, CSA2_DEVERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t phase, int32_t *err) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait1(bar, phase, err) ? 1 : 0;
  if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
  tc::mbar_wait_bounded(bar, phase, kWaitIters);  // (each lane observes the phase itself)
  return true;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(kN) : "memory");
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

// kQuery: K = dim in one stage, W [dim][np] read MN-major.  Value: K = 512 in stages of
// kKc columns (fp32: hi and lo), W [np][512] K-major.
template <bool kQuery, bool kF32>
struct Shape {
  static constexpr int kStageBytes = kQuery ? kTok * 128 * 2 : kTok * 64 * 2;
  static constexpr int kStages = kQuery ? 2 : 5;
  static constexpr int kKc = kQuery ? 128 : kF32 ? 32 : 64;
  static constexpr int kBytes = kWBytesMax + kStages * kStageBytes + 1024;
};

template <bool kQuery, bool kF32>
__global__ void __launch_bounds__(kThreads, 1) k_latent(LatentArgs a) {
  using S = Shape<kQuery, kF32>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) Sync sy;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t s_w = (tc::smem_addr(raw) + 1023) & ~1023u, s_x = s_w + kWBytesMax;
  const int jobs = kQuery && a.np > 256 ? 2 : 1, cols = a.np / jobs;  // accumulators of a unit, their columns
  const int chunks = kQuery ? 1 : kLat / S::kKc;
  const int w_rows = kQuery ? a.dim : a.np;                          // rows of W in shared memory
  const int64_t units = static_cast<int64_t>(a.heads) * a.parts * a.tiles;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  if (warp == kIssueWarp) {
    tc::tmem_alloc(&sy.tmem, 512);
    tc::tmem_relinquish();
  }
  if (t == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      tc::mbar_init(&sy.full[i], kLoadWarps);
      tc::mbar_init(&sy.empty[i], 1);
    }
    tc::mbar_init(&sy.wfull, kLoadWarps);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sy.tfull[i], 1);
      tc::mbar_init(&sy.tempty[i], 4);
    }
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sy.tmem;

  if (warp < kLoadWarps) {
    // ------------------------------------------------------------ loads
    const int r8 = lane & 7, uo = lane >> 3;  // row in a group of 8, 16-byte unit of four
    int64_t held = -1;
    uint32_t n = 0;        // stages filled so far
    uint32_t pending = 0;  // ... whose hand-over is still to come
    bool ok = true;
    auto hand_over = [&](uint64_t *bar) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    for (int64_t u = u0; u < u1 && ok; ++u) {
      const int64_t hp = u / a.tiles;
      const int tile = static_cast<int>(u - hp * a.tiles), h = static_cast<int>(hp / a.parts), part = static_cast<int>(hp % a.parts);
      const int t0 = tile * kTok, rows = min(kTok, a.total - t0);
      if (hp != held) {
        for (; pending > 0; --pending) {
          cp_wait<0>();
          hand_over(&sy.full[(n - pending) % S::kStages]);
        }
        // W is free once the last stage's MMAs are done
        if (n > 0) ok = wait_warp(&sy.empty[(n - 1) % S::kStages], ((n - 1) / S::kStages) & 1, a.err);
        if (!ok) break;
        const uint16_t *src = a.w + h * a.w_stride + (kQuery ? part * a.np : static_cast<int64_t>(part) * a.np * kLat);
        const int w_units = (kQuery ? a.np : kLat) / 8;
        for (int i = warp; i < (w_rows / 8) * (w_units / 4); i += kLoadWarps) {
          const int rg = i % (w_rows / 8), un = 4 * (i / (w_rows / 8)) + uo;
          cp16(s_w + un * (w_rows * 16) + rg * 128 + r8 * 16, src + static_cast<int64_t>(8 * rg + r8) * kLat + 8 * un);
        }
        cp_commit();
        cp_wait<0>();
        hand_over(&sy.wfull);
        held = hp;
      }
      for (int c = 0; c < chunks && ok; ++c, ++n) {
        const int st = n % S::kStages;
        if (n >= S::kStages) ok = wait_warp(&sy.empty[st], ((n / S::kStages) - 1) & 1, a.err);
        if (!ok) break;
        const uint32_t dst = s_x + st * S::kStageBytes;
        if constexpr (!kF32) {
          const uint16_t *src = static_cast<const uint16_t *>(a.x) + t0 * a.x_stride +
                                (kQuery ? static_cast<int64_t>(h) * (a.dim + kRope) : static_cast<int64_t>(h) * kLat + c * S::kKc);
          const int n_un = kQuery ? a.dim / 8 : S::kKc / 8, quads = (n_un + 3) / 4;
          for (int i = warp; i < 16 * quads; i += kLoadWarps) {
            const int r = 8 * (i % 16) + r8, un = 4 * (i / 16) + uo;
            if (r < rows && un < n_un) cp16(dst + un * (kTok * 16) + r * 16, src + r * a.x_stride + 8 * un);
          }
          cp_commit();
          ++pending;
          if constexpr (!kQuery) {  // three stages in flight
            if (pending == 3) {
              cp_wait<2>();
              hand_over(&sy.full[(n - 2) % S::kStages]);
              --pending;
            }
          }
        } else {
          const float *src = static_cast<const float *>(a.x) + t0 * a.x_stride + static_cast<int64_t>(h) * kLat + c * S::kKc;
          float4 v[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * (warp + 8 * i) + r8;
            v[i][0] = v[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows) {
              const float4 *p = reinterpret_cast<const float4 *>(src + r * a.x_stride + 8 * uo);
              v[i][0] = __ldg(p);
              v[i][1] = __ldg(p + 1);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * (warp + 8 * i) + r8;
            uint32_t hi[4], lo[4];
            split2(v[i][0].x, v[i][0].y, hi[0], lo[0]);
            split2(v[i][0].z, v[i][0].w, hi[1], lo[1]);
            split2(v[i][1].x, v[i][1].y, hi[2], lo[2]);
            split2(v[i][1].z, v[i][1].w, hi[3], lo[3]);
            const uint32_t at = dst + uo * (kTok * 16) + r * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at + 8192), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
          }
          hand_over(&sy.full[st]);
        }
      }
      if constexpr (kQuery) {
        if (!ok) break;
        // RoPE while the rows arrive: a thread takes 8 dims of a token
        if (part == 0) {
          const uint16_t *qr = static_cast<const uint16_t *>(a.x) + static_cast<int64_t>(h) * (a.dim + kRope) + a.dim;
          for (int i = warp; i < kTok / 4; i += kLoadWarps) {
            const int r = 4 * i + uo, d8 = r8;
            if (r >= rows) continue;
            const int64_t tok = t0 + r, p = a.pos[tok];
            if (p < 0) continue;
            if (p >= a.rope_len) {
              if (h == 0 && d8 == 0) raise_err(a.err, CSA2_DEVERR_ROPE);
              continue;
            }
            rotate8(a, qr + tok * a.x_stride + 8 * d8, p, d8, a.out + tok * a.out_stride + static_cast<int64_t>(h) * kDqk + kLat + 8 * d8);
          }
        }
        cp_wait<0>();
        hand_over(&sy.full[(n - 1) % S::kStages]);
        pending = 0;
      }
    }
    cp_wait<0>();
    if (ok)
      for (; pending > 0; --pending) hand_over(&sy.full[(n - pending) % S::kStages]);
  } else if (warp == kIssueWarp) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0) {
      const uint32_t id = idesc_bf16(cols, kQuery ? 1 : 0);
      const uint32_t wu = w_rows * 16;  // bytes from one 8-column unit of W to the next
      int64_t held = -1;
      uint32_t n = 0, j = 0, wn = 0;
      bool ok = true;
      for (int64_t u = u0; u < u1 && ok; ++u) {
        const int64_t hp = u / a.tiles;
        if (hp != held) {
          ok = wait1(&sy.wfull, wn++ & 1, a.err);
          held = hp;
          if (!ok) break;
        }
        for (int b = 0; b < jobs && ok; ++b, ++j) {
          const uint32_t acc = j & 1, d = tmem + 256 * acc;
          if (j >= 2) ok = wait1(&sy.tempty[acc], ((j >> 1) - 1) & 1, a.err);
          for (int c = 0; c < chunks && ok; ++c) {
            const uint32_t k = kQuery ? n : n + c, st = k % S::kStages;
            if (b == 0) ok = wait1(&sy.full[st], (k / S::kStages) & 1, a.err);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t xa = s_x + st * S::kStageBytes;
            if constexpr (kQuery) {
              for (int s = 0; s < a.dim / 16; ++s)
                mma_bf16(d, tc::smem_desc_noswizzle(xa + 4096 * s, 2048, 128),
                         tc::smem_desc_noswizzle(s_w + b * (cols / 8) * wu + 256 * s, 128, wu), id, s > 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int s = 0; s < S::kKc / 16; ++s) {
                const uint64_t wd = tc::smem_desc_noswizzle(s_w + (c * (S::kKc / 8) + 2 * s) * wu, wu, 128);
                mma_bf16(d, tc::smem_desc_noswizzle(xa + 4096 * s, 2048, 128), wd, id, c + s > 0 ? 1u : 0u);
                if constexpr (kF32) mma_bf16(d, tc::smem_desc_noswizzle(xa + 8192 + 4096 * s, 2048, 128), wd, id, 1u);
              }
            }
            if (b == jobs - 1) tc::mma_commit(&sy.empty[st]);
          }
          if (ok) tc::mma_commit(&sy.tfull[acc]);
        }
        n += chunks;
      }
    }
  } else {
    // ------------------------------------------------------------ results
    const int q = warp & 3, g = (warp - kLoadWarps) >> 2;
    uint32_t j = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok; ++u) {
      const int64_t hp = u / a.tiles;
      const int tile = static_cast<int>(u - hp * a.tiles), h = static_cast<int>(hp / a.parts), part = static_cast<int>(hp % a.parts);
      const int64_t tok = static_cast<int64_t>(tile) * kTok + 32 * q + lane;
      for (int b = 0; b < jobs && ok; ++b, ++j) {
        if ((j & 1) != g) continue;
        bool live = tok < a.total;
        if constexpr (kQuery) {
          if (live) {
            const int64_t p = a.pos[tok];
            live = p >= 0 && p < a.rope_len;
          }
        }
        uint16_t *dst = a.out + tok * a.out_stride + (kQuery ? static_cast<int64_t>(h) * kDqk : static_cast<int64_t>(h) * a.dim) +
                        part * a.np + b * cols;
        ok = wait_warp(&sy.tfull[g], (j >> 1) & 1, a.err);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t at = tmem + 256 * g + (static_cast<uint32_t>(32 * q) << 16);
        for (int c = 0; c < cols; c += 16) {
          uint32_t r[16];
          tc::tmem_ld_32x32b_x16(at + c, r);
          tc::tmem_ld_wait_x16(r);
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
          if (live) {
            if (a.wide) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + c), "r"(o[0]), "r"(o[1]),
                           "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                           : "memory");
            } else {
              reinterpret_cast<uint4 *>(dst + c)[0] = make_uint4(o[0], o[1], o[2], o[3]);
              reinterpret_cast<uint4 *>(dst + c)[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sy.tempty[g]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <bool kQuery, bool kF32>
cudaError_t launch(const LatentArgs &a, cudaStream_t s) {
  const auto kern = k_latent<kQuery, kF32>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kern), Shape<kQuery, kF32>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.heads) * a.parts * a.tiles, sms = device_sm_count();
  kern<<<static_cast<unsigned>(units < sms ? units : sms), kThreads, Shape<kQuery, kF32>::kBytes, s>>>(a);
  return cudaGetLastError();
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
  const int64_t units = static_cast<int64_t>(n_heads) * a.tiles, sms = csa2::device_sm_count();
  a.parts = 2 * units > sms ? 1 : 4 * units > sms ? 2 : 4;
  a.np = CSA2_D_LATENT / a.parts;
  a.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  a.err = err_word;
  if (total <= csa2::kFewTokens)
    return cuda_status(csa2::launch_query_few(a, reinterpret_cast<cudaStream_t>(stream)), "csa2_query_latent launch");
  return cuda_status(csa2::launch<true, false>(a, reinterpret_cast<cudaStream_t>(stream)), "csa2_query_latent launch");
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
  const int64_t units = static_cast<int64_t>(n_heads) * a.tiles, sms = csa2::device_sm_count();
  a.parts = 1;
  while (2 * units * a.parts <= sms && dim % (32 * a.parts) == 0 && a.parts < 4) a.parts *= 2;
  a.np = dim / a.parts;
  a.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && out_stride % 16 == 0;
  a.err = err_word;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (total <= csa2::kFewTokens)
    return cuda_status(csa2::launch_value_few(a, in_dtype == CSA2_IN_F32, s), "csa2_value_project launch");
  return cuda_status(in_dtype == CSA2_IN_F32 ? csa2::launch<false, true>(a, s) : csa2::launch<false, false>(a, s),
                     "csa2_value_project launch");
}

}  // extern "C"
