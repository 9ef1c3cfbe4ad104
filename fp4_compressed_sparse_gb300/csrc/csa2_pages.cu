// csa2_pages.cu -- the pages of a paged cache handed out on the GPU from the
// sequences' lengths (csa2_pages_resize), and where each new token of a ragged
// batch will lie (csa2_slot_map).
//
// Pages ([P5] "DeepSeek-V4: Towards Highly Efficient Million-Token Context
// Intelligence" §3.5.1, blocks of a multiple of lcm(m, m') tokens).  Sequence b
// needs need_b = ceil(floor(n_b / ratio) / page_entries) pages.  Free pages are a
// stack.  With R the pages that sequences give back and n0 the free ones before, the
// j-th of them (in sequence and page order) goes to free[n0 + R - 1 - j], and the
// k-th page that is taken comes from free[n0 + R - 1 - k]: two exclusive prefix sums
// give every move its place, so there is no atomic, equal calls give equal tables, and
// giving pages back undoes taking them.
//
// Bound: latency.  A decode step of 32 sequences reads a few hundred bytes; what it
// takes is the chain lengths -> prefix sum -> barrier -> free list -> table.  32 sequences
// that keep their pages 2.9 us, a launch alone 1.4; that take a page each and give it back
// 4.5 a call, 499 pages each 11.2; 512, of which 51 end and 51 bring prompts, and back 8.7 a
// call (the look at what comes back: 1.5, 6 and 4 us of two such calls).  The slots of 32 and of
// 104,034 tokens 2.6 and 4.2.
#include "csa2_internal.cuh"

namespace csa2 {
namespace {

constexpr int kPageThreads = 1024;
// one cluster: 32 sequences that take or give 499 pages each 11.2 us, with one CTA 62; one
// page each 4.5, with one CTA 4.3
constexpr int kPageCtas = 8;
constexpr int kMaskWords = 65536 / 32;  // a bit per sequence

struct PagesArgs {
  csa2_cache c;
  int32_t *table;  // c.block_table
  csa2_page_pool pool;
  const int64_t *target;
  const int32_t *cu;
  int total, max_new;
  int32_t *granted;
  int32_t *err;
};

// What sequence b holds and needs; ok false: broken or too long, left as it is.
struct SeqPages {
  int held, need;
  bool ok;
};
struct SeqIn {
  int held;
  int64_t n;  // the target, or the tokens before the step
};
__device__ __forceinline__ SeqIn seq_in(const PagesArgs &a, int b) {
  return SeqIn{a.pool.held[b], a.target != nullptr ? a.target[b] : a.c.n_tokens[b]};
}
__device__ __forceinline__ SeqPages seq_pages(const PagesArgs &a, int b, SeqIn in, int falls, bool report) {
  SeqPages s{in.held, 0, false};
  bool good = s.held >= 0 && s.held <= a.c.max_pages;
  int64_t n = in.n;
  if (a.target == nullptr) {
    good = good && n >= 0;
    if (a.cu != nullptr) {
      int first, cnt;
      good = ragged_rows(a.cu, b, a.total, a.max_new, first, cnt) && good;
      if (falls && cnt > 0) good = ragged_own(a.cu, a.c.batch, b, first, cnt) && good;
      n += cnt;
    }
  }
  good = good && n >= 0;
  const int64_t ent = n / a.c.ratio;
  s.ok = good && ent <= a.c.capacity;
  if (report && !s.ok) raise_err(a.err, good ? CSA2_DEVERR_CAPACITY : CSA2_DEVERR_INDEX);
  s.need = s.ok ? static_cast<int>((ent + a.c.page_entries - 1) / a.c.page_entries) : s.held;
  return s;
}

// Inclusive sums of x and y over the block, and the totals.
struct Scan2 {
  int64_t x, y, x_all, y_all;
};
__device__ __forceinline__ Scan2 block_scan2(int64_t x, int64_t y, int64_t (*sh)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  __syncthreads();  // (sh may still be read from the scan before)
  if (lane == 31) {
    sh[warp][0] = x;
    sh[warp][1] = y;
  }
  __syncthreads();
  Scan2 r{x, y, 0, 0};
  for (int w = 0; w < nw; ++w) {
    if (w < warp) {
      r.x += sh[w][0];
      r.y += sh[w][1];
    }
    r.x_all += sh[w][0];
    r.y_all += sh[w][1];
  }
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// The 32 bits at the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t peer_word(const void *p, int rank) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// First t in [0, n) with list[t] > v (list non-decreasing, list[n - 1] > v).
__device__ __forceinline__ int first_above(const int64_t *list, int n, int64_t v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (list[mid] > v) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// One cluster.  Every CTA computes all prefix sums (a chunk of blockDim sequences at a
// time) and moves every gridDim-th page, so what passes between them is the barriers and,
// where pages come back, the sequences whose ids are no pages: those are looked for before
// anything is written, since whoever grew would get such an id from the stack.  free and
// table: written between the barriers; held, granted and n_free, which every CTA reads,
// behind the last.
__global__ void __launch_bounds__(kPageThreads) k_pages_resize(PagesArgs a) {
  __shared__ int64_t sh[32][2];
  __shared__ int64_t l_back[kPageThreads], l_grow[kPageThreads];
  __shared__ int32_t l_held[kPageThreads], l_need[kPageThreads];
  __shared__ uint32_t found[kMaskWords], broken[kMaskWords];  // a bit per sequence: this CTA's finds, all CTAs'
  __shared__ uint32_t any_found;
  const int t = threadIdx.x, nthr = blockDim.x, rank = blockIdx.x, ctas = gridDim.x;
  const int batch = a.c.batch, mp = a.c.max_pages;
  for (int w = t; w < (batch + 31) / 32; w += nthr) found[w] = broken[w] = 0;
  next_may_start();
  wait_for_previous();
  const int64_t n0 = *a.pool.n_free;
  const bool one = batch <= nthr;
  SeqIn in{0, 0};
  if (one && t < batch) in = seq_in(a, t);  // (on its way while the bounds are read)
  int falls = 0;
  if (a.cu != nullptr)
    for (int b = t; b < batch; b += nthr) falls |= a.cu[b + 1] < a.cu[b];
  falls = __syncthreads_or(falls);

  SeqPages s{0, 0, false};
  Scan2 c{};
  int64_t R = 0;
  auto seq = [&](int b, SeqIn in, bool report) {
    SeqPages x = seq_pages(a, b, in, falls, report);
    if (broken[b >> 5] >> (b & 31) & 1) x.need = x.held, x.ok = false;
    return x;
  };
  // pages that go back, altogether (one chunk: s and c stay for what follows)
  auto count = [&](bool report) {
    if (one) {
      if (t < batch) s = seq(t, in, report);
      c = block_scan2(max(s.held - s.need, 0), max(s.need - s.held, 0), sh);
      R = c.x_all;
    } else {
      int64_t mine = 0;
      for (int b = t; b < batch; b += nthr) {
        s = seq(b, seq_in(a, b), report);
        mine += max(s.held - s.need, 0);
      }
      R = block_scan2(mine, 0, sh).x_all;
    }
  };
  // each of them, dealt to the cluster's threads: its place in sequence and page order, its sequence, its entry
  auto each_back = [&](auto use) {
    int64_t base = 0;
    for (int b0 = 0; b0 < batch; b0 += nthr) {
      if (!one) {
        s = b0 + t < batch ? seq(b0 + t, seq_in(a, b0 + t), false) : SeqPages{0, 0, false};
        c = block_scan2(max(s.held - s.need, 0), 0, sh);
      }
      l_back[t] = c.x;
      l_held[t] = s.held;
      l_need[t] = s.need;
      __syncthreads();
      for (int64_t j = static_cast<int64_t>(rank) * nthr + t; j < c.x_all; j += static_cast<int64_t>(ctas) * nthr) {
        const int q = first_above(l_back, nthr, j);
        const int p = l_need[q] + static_cast<int>(j - (l_back[q] - (l_held[q] - l_need[q])));
        use(base + j, b0 + q, a.table + static_cast<int64_t>(b0 + q) * mp + p);
      }
      base += c.x_all;
      __syncthreads();
    }
  };
  count(rank == 0);
  if (R > 0) {  // (the same in every thread of the cluster)
    int mine = 0;
    each_back([&](int64_t, int b, const int32_t *e) {
      if (*e >= 0 && *e < a.c.n_pages) return;
      atomicOr(&found[b >> 5], 1u << (b & 31));
      mine = 1;
    });
    if (mine) raise_err(a.err, CSA2_DEVERR_INDEX);
    mine = __syncthreads_or(mine);
    if (t == 0) any_found = mine;
    cluster_sync();
    if (__syncthreads_or(t < ctas ? peer_word(&any_found, t) : 0u)) {
      for (int w = t; w < (batch + 31) / 32; w += nthr) {
        uint32_t m = 0;
        for (int r = 0; r < ctas; ++r) m |= peer_word(&found[w], r);
        broken[w] = m;
      }
      __syncthreads();
      count(false);
    }
  }
  const int64_t n1 = n0 + R;
  const bool sound = n0 >= 0 && n1 <= a.c.n_pages;  // (the same in every thread of the cluster)
  if (!sound && rank == 0 && t == 0) raise_err(a.err, CSA2_DEVERR_INDEX);

  // ---- pages back to the stack
  if (sound && R > 0)
    each_back([&](int64_t j, int, int32_t *e) {
      a.pool.free[n1 - 1 - j] = *e;
      *e = -1;
    });
  cluster_sync();

  // ---- pages from the stack, as long as a sequence's whole need fits
  int64_t taken = 0, base = 0;
  for (int b0 = 0; b0 < batch && sound; b0 += nthr) {
    const int b = b0 + t;
    if (!one) {
      s = b < batch ? seq(b, seq_in(a, b), false) : SeqPages{0, 0, false};
      c = block_scan2(0, max(s.need - s.held, 0), sh);
    }
    const int64_t fit = n1 - base;  // what the chunk may take
    l_grow[t] = c.y;
    l_held[t] = s.held;
    l_need[t] = s.need;
    __syncthreads();
    const int64_t last = min(c.y_all, fit);
    for (int64_t k = static_cast<int64_t>(rank) * nthr + t; k < last; k += static_cast<int64_t>(ctas) * nthr) {
      const int q = first_above(l_grow, nthr, k);
      if (l_grow[q] > fit) continue;  // the sequence's pages do not all fit: none
      const int p = l_held[q] + static_cast<int>(k - (l_grow[q] - (l_need[q] - l_held[q])));
      a.table[static_cast<int64_t>(b0 + q) * mp + p] = a.pool.free[n1 - 1 - (base + k)];
    }
    // the largest sum that still fits is what the stack loses
    int64_t top = c.y <= fit ? c.y : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if ((t & 31) == 0) sh[t >> 5][0] = top;
    __syncthreads();
    top = 0;
    for (int w = 0; w < (nthr >> 5); ++w) top = max(top, sh[w][0]);
    taken = top > 0 ? base + top : taken;
    base += c.y_all;
    __syncthreads();
  }
  cluster_sync();

  // ---- counts
  if (rank != 0) return;
  base = 0;
  for (int b0 = 0; b0 < batch; b0 += nthr) {
    const int b = b0 + t;
    if (!one) {  // (held[b] is still the old one: this thread writes it next)
      s = b < batch ? seq(b, seq_in(a, b), false) : SeqPages{0, 0, false};
      c = block_scan2(0, max(s.need - s.held, 0), sh);
    }
    if (b < batch) {
      const bool has = s.ok && sound && (s.need <= s.held || base + c.y <= n1);
      if (has && s.need != s.held) a.pool.held[b] = s.need;
      if (a.granted != nullptr) a.granted[b] = has ? 1 : 0;
    }
    base += c.y_all;
  }
  if (t == 0 && sound) *a.pool.n_free = static_cast<int32_t>(n1 - taken);
}

// One thread per packed row: its sequence (a binary search in cu), position and entry.
__global__ void __launch_bounds__(256) k_slot_map(csa2_cache c, const int32_t *cu, int total, int max_new, int64_t *slots,
                                                  int64_t *pos, int32_t *err) {
  next_may_start();
  wait_for_previous();
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r < c.batch) {  // every broken list shows in some sequence's bounds
    int first, n;
    if (!ragged_rows(cu, r, total, max_new, first, n)) raise_err(err, CSA2_DEVERR_INDEX);
  }
  if (r >= total) return;
  const RaggedRow x = ragged_row(cu, c.batch, total, max_new, r);
  int64_t slot = -1, p = -1;
  if (x.b >= 0 && x.n > 0) {
    const int64_t t0 = c.n_tokens[x.b], t = t0 + (r - x.first), e = t / c.ratio;
    if (t0 >= 0) {
      p = t;
      if (e < (t0 + x.n) / c.ratio) {
        if (e >= c.capacity) {
          raise_err(err, CSA2_DEVERR_CAPACITY);
        } else {
          slot = phys_entry(entry_map(c), x.b, e);
          if (slot < 0) raise_err(err, CSA2_DEVERR_INDEX);
        }
      }
    } else {
      raise_err(err, CSA2_DEVERR_INDEX);
    }
  }
  if (slots != nullptr) slots[r] = slot;
  if (pos != nullptr) pos[r] = p;
}

}  // namespace
}  // namespace csa2

extern "C" {

using csa2::check_cache;
using csa2::cuda_status;

csa2_status csa2_pages_resize(const csa2_cache *cache, const csa2_page_pool *pool, const int64_t *target,
                              const int32_t *cu_new, int32_t total, int32_t max_new, int32_t *granted, int32_t *err_word,
                              csa2_stream_t stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE(cache->block_table != nullptr, CSA2_ERR_NULL, "block_table is NULL: a dense cache has no pages");
  CSA2_REQUIRE(pool != nullptr, CSA2_ERR_NULL, "pool is NULL");
  CSA2_REQUIRE_PTR(pool->free);
  CSA2_REQUIRE_PTR(pool->n_free);
  CSA2_REQUIRE_PTR(pool->held);
  CSA2_REQUIRE_OPT_PTR(target);
  CSA2_REQUIRE_OPT_PTR(cu_new);
  CSA2_REQUIRE_OPT_PTR(granted);
  CSA2_REQUIRE(target == nullptr || cu_new == nullptr, CSA2_ERR_RANGE, "target and cu_new are both given");
  CSA2_REQUIRE(total >= 0 && total <= (1 << 24), CSA2_ERR_SHAPE, "total %d outside 0..2^24", total);
  CSA2_REQUIRE(max_new >= 0, CSA2_ERR_SHAPE, "max_new %d < 0", max_new);
  csa2::PagesArgs a{*cache, const_cast<int32_t *>(cache->block_table), *pool, target, cu_new, total, max_new, granted, err_word};
  const int threads = cache->batch >= csa2::kPageThreads ? csa2::kPageThreads : (cache->batch + 31) / 32 * 32;
  const int block = threads < 256 ? 256 : threads;
  return cuda_status(csa2::launch_after(csa2::k_pages_resize, dim3(csa2::kPageCtas), block, 0, csa2::kPageCtas,
                                        reinterpret_cast<cudaStream_t>(stream), a),
                     "csa2_pages_resize launch");
}

csa2_status csa2_slot_map(const csa2_cache *cache, const int32_t *cu_new, int32_t total, int32_t max_new, int64_t *slots,
                          int64_t *pos, int32_t *err_word, csa2_stream_t stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  CSA2_REQUIRE_PTR(cu_new);
  CSA2_REQUIRE(total >= 0 && total <= (1 << 24), CSA2_ERR_SHAPE, "total %d outside 0..2^24", total);
  CSA2_REQUIRE(max_new >= 0, CSA2_ERR_SHAPE, "max_new %d < 0", max_new);
  CSA2_REQUIRE(slots != nullptr || pos != nullptr, CSA2_ERR_NULL, "slots and pos are both NULL");
  CSA2_REQUIRE_OPT_PTR(slots);
  CSA2_REQUIRE_OPT_PTR(pos);
  if (total == 0) return CSA2_OK;
  const int n = total > cache->batch ? total : cache->batch;
  return cuda_status(csa2::launch_after(csa2::k_slot_map, dim3((n + 255) / 256), 256, 0, 0, reinterpret_cast<cudaStream_t>(stream), *cache,
                                        cu_new, total, max_new, slots, pos, err_word),
                     "csa2_slot_map launch");
}

}  // extern "C"
