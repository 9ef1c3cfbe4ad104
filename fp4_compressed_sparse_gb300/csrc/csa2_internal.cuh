// csa2_internal.cuh -- launchers shared between the libcsa2 translation units.
#pragma once

#include "csa2_device.cuh"

namespace csa2 {

// ------------------------------------------------------------------ host helpers (csa2_api.cu)
// thread-local text returned by csa2_last_error_detail()
void set_error_detail(const char *msg);
// records a printf-style detail for csa2_last_error_detail() and returns st
csa2_status fail(csa2_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// CSA2_OK for cudaSuccess, else CSA2_ERR_CUDA with "what: <CUDA error text>" as the detail
csa2_status cuda_status(cudaError_t e, const char *what);
// host validation of a cache descriptor
csa2_status check_cache(const csa2_cache *c);
// host validation of a 4-bit matrix (csa2_fp4.cu); name: its argument's
csa2_status check_fp4(const csa2_fp4_matrix *m, const char *name);
// SM count of the current device (queried once per device)
int device_sm_count();
// Raises fn's dynamic shared-memory limit to at least `bytes` on the current
// device (the attribute is per device: set once per (device, kernel)).
cudaError_t ensure_smem_limit(const void *fn, int bytes);

__host__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define CSA2_REQUIRE(cond, status, ...)                  \
  do {                                                   \
    if (!(cond)) return ::csa2::fail(status, __VA_ARGS__); \
  } while (0)

#define CSA2_REQUIRE_PTR(p)                                                                 \
  do {                                                                                      \
    if ((p) == nullptr) return ::csa2::fail(CSA2_ERR_NULL, "%s is NULL", #p);               \
    if (!::csa2::aligned16(p)) return ::csa2::fail(CSA2_ERR_ALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)

#define CSA2_REQUIRE_OPT_PTR(p)                                                             \
  do {                                                                                      \
    if ((p) != nullptr && !::csa2::aligned16(p))                                            \
      return ::csa2::fail(CSA2_ERR_ALIGN, "%s is not 16-byte aligned", #p);                 \
  } while (0)

// ------------------------------------------------------------------ overlapped launches
// A kernel launched by launch_after() may be resident and set itself up while the kernel
// before it in the stream drains (or, once all blocks of that one have called
// next_may_start(), while it runs).  It calls wait_for_previous() in every thread before it
// reads or writes anything in memory.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// Loads of what a kernel before may have written, for kernels launched so: not through the
// read-only path (the memory changes while such a kernel is resident), and volatile, which
// keeps them behind wait_for_previous() and lets them pass the kernel's own stores.
__device__ __forceinline__ uint4 load_now(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(__cvta_generic_to_global(p)));
  return v;
}
__device__ __forceinline__ float4 load_now(const float4 *p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(__cvta_generic_to_global(p)));
  return v;
}
__device__ __forceinline__ uint2 load_now(const uint2 *p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(__cvta_generic_to_global(p)));
  return v;
}
__device__ __forceinline__ uint32_t load_now(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];\n" : "=r"(v) : "l"(__cvta_generic_to_global(p)));
  return v;
}
template <class... P, class... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int block, size_t smem, int cluster, cudaStream_t s, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

cudaError_t launch_kv_append(const csa2_cache &c, const void *kv, const void *ik, int in_dtype,
                             const csa2_compress_in *cmp, const float *rope_cs, int64_t rope_len, int n_new,
                             float *cmp_dbg, int32_t *err, cudaStream_t s);

// ------------------------------------------------------------------ ragged batches
// Rows of sequence b: its first row and their number; false (count 0) when cu is
// not a non-decreasing list within 0..total, or the count breaks max_new.
__device__ __forceinline__ bool ragged_rows(const int32_t *cu, int b, int total, int max_new, int &first, int &n) {
  first = cu[b];
  const int end = cu[b + 1];
  const bool ok = first >= 0 && end >= first && end <= total && end - first <= max_new;
  n = ok ? end - first : 0;
  return ok;
}
// The sequence of packed row r by a binary search (b -1: a row of no sequence), with
// its rows as ragged_rows gives them.  n is 0 as well when the search met a bound on
// its way that does not lie before or after those rows: the list decreases somewhere,
// and the rows may be another sequence's too.  The way to b is the same for every row
// that leads there, so a sequence's rows agree, and the rows of two sequences that
// pass lie apart (where their ways part, one bound is behind the one's and before the
// other's).
struct RaggedRow {
  int b, first, n;
};
__device__ __forceinline__ RaggedRow ragged_row(const int32_t *cu, int batch, int total, int max_new, int r) {
  RaggedRow x{-1, cu[0], 0};
  int end = cu[batch];
  if (r >= end || r < x.first) return x;
  int lo = 0, hi = batch, below = x.first, above = end;  // cu[lo] = x.first <= r < cu[hi] = end
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, v = cu[mid];
    if (v <= r) {
      lo = mid;
      x.first = v;
      below = max(below, v);
    } else {
      hi = mid;
      end = v;
      above = min(above, v);
    }
  }
  x.b = lo;
  if (x.first >= 0 && end <= total && end - x.first <= max_new && below == x.first && above == end) x.n = end - x.first;
  return x;
}
// Whether ragged_row would give rows first .. first + n - 1 to sequence b: bound number
// `step` of the way there (0 and 1: the list's ends), true behind its end.
__device__ __forceinline__ bool ragged_own_step(const int32_t *cu, int batch, int b, int first, int n, int step) {
  if (step == 0) return cu[0] <= first;
  if (step == 1) return cu[batch] >= first + n;
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (--step == 1) return mid <= b ? cu[mid] <= first : cu[mid] >= first + n;
    if (mid <= b) lo = mid;
    else hi = mid;
  }
  return true;
}
constexpr int kOwnSteps = 18;  // of a batch of 65,535
// ... all of them, by one thread (few loads wait for one another).
__device__ __forceinline__ bool ragged_own(const int32_t *cu, int batch, int b, int first, int n) {
  bool ok = true;
  for (int step = 0; step < kOwnSteps; ++step) ok = ragged_own_step(cu, batch, b, first, n, step) && ok;
  return ok;
}
// ... all of them, by the block, a thread for each (a barrier).
__device__ __forceinline__ bool block_ragged_own(const int32_t *cu, int batch, int b, int first, int n) {
  const int t = threadIdx.x;
  return __syncthreads_and(t >= kOwnSteps || ragged_own_step(cu, batch, b, first, n, t));
}

// ------------------------------------------------------------------ score sideband
// Per score row, the index-score kernel also leaves a 13-bit histogram of the
// order-preserving score keys and (FULL rows) the maxima of 8-position blocks
// with their histogram; the selector reads these instead of re-scanning.
// Row layout: hist[0][kSelBins] (scores) | hist[1][kSelBins] (block maxima) |
// bmax[ceil(stride/8)] floats, padded to 16 bytes.
constexpr int kSelBins = 8192;
constexpr int kSelBinShift = 19;  // key >> 19 = top 13 bits
constexpr int kSelCap = 4096;     // candidates kept per (row, problem)
__host__ __device__ __forceinline__ int64_t aux_row_bytes(int64_t stride) {
  return 2 * kSelBins * 4 + ((((stride + 7) / 8) * 4 + 15) / 16) * 16;
}

// ------------------------------------------------------------------ index score
struct ScoreArgs {
  const uint8_t *idx_codes;   // cache plane base
  const uint8_t *idx_scales;
  EntryMap map;               // where a sequence's entries live (dense or paged)
  int64_t cap;                // entries per sequence
  int ratio;
  int rows;                   // query rows
  int heads;                  // H_I
  const uint16_t *q_idx;      // [rows][H_I][128] bf16
  const float *w;             // [rows][H_I]
  const int64_t *q_pos;       // [rows]
  int cache_seq;              // -1: row r reads sequence r; else every row reads this sequence
  const int32_t *pool;        // POOL mode: [rows][pool_blocks]; nullptr = FULL
  int pool_blocks, pool_bs;
  float *scores;              // [rows][stride]
  int64_t stride;
  uint8_t *aux;               // [rows][aux_row_bytes(stride)] sideband (its histograms are cleared by the launch), or nullptr
  int32_t *err;
  int no_block_max;           // FULL with aux: 1 = the score histogram alone (no pool will be built from it)
};
cudaError_t launch_index_score(const ScoreArgs &a, cudaStream_t s);  // CUDA cores (dp4a), no sideband
// tensor cores (tcgen05 kind::mxf4); needs pool == nullptr or pool_bs == 8, heads <= 128; fills aux
size_t score_tc_workspace_bytes(int rows, int heads);
cudaError_t launch_index_score_tc(const ScoreArgs &a, void *ws, cudaStream_t s);

// ------------------------------------------------------------------ top-k
struct TopkArgs {
  int rows;
  const float *scores;        // [rows][stride]
  int64_t stride;
  const uint8_t *aux;         // sideband from the score kernel, or nullptr (built here)
  int ratio;
  const int64_t *q_pos;       // [rows]
  const int32_t *pool;        // POOL rows: [rows][pool_blocks] ascending block ids; nullptr = FULL
  int pool_blocks, bs;
  int k;
  int32_t *idx_out;           // [rows][k]
  int out_pool_blocks;        // FULL only: candidate-pool size (0 = no pool)
  int32_t *pool_out;          // [rows][out_pool_blocks]
  int32_t *pool_count;        // [rows]
  int32_t *err;
};
size_t topk_workspace_bytes(int rows, int64_t stride, bool have_aux);
// fills the sideband of `rows` score rows from the scores themselves
cudaError_t launch_fill_aux(const TopkArgs &a, uint8_t *aux, cudaStream_t s);
cudaError_t launch_topk(const TopkArgs &a, void *ws, cudaStream_t s);

// ------------------------------------------------------------------ attention
struct AttnArgs {
  int rows, heads, k;
  const uint16_t *q;          // [rows][H][576]
  const int32_t *idx;         // [rows][k]
  const int64_t *q_pos;       // [rows]
  int cache_seq;              // -1: row = sequence
  const uint8_t *lat_codes, *lat_scales, *rope_codes, *rope_scales;
  EntryMap map;               // where a sequence's entries live (dense or paged)
  int entry_format;           // CSA2_ENTRY_FP4 or CSA2_ENTRY_FP8
  int64_t cap;
  int ratio;
  const int64_t *n_tokens;    // [batch]
  const uint8_t *ring_codes, *ring_scales;  // window ring [seq][128][...]
  int ring_single;            // 1: the ring holds only cache_seq's 128 slots
  int swa_dtype;
  const uint8_t *lin_codes, *lin_scales;    // window tokens >= *lin_base: [t - *lin_base][...]
  const int64_t *lin_base;    // device scalar or nullptr
  const float *sink;          // [H] or nullptr
  float sm_scale;
  float *out, *lse;
  int32_t *err;
};
// Segments of a decode row (a function of k alone: the batch-invariant
// accumulation order); a row's output is the ordered merge of its segments.
int attn_segments(int k);
size_t attn_workspace_bytes(int rows, int heads, int n_seg);
cudaError_t launch_attn(const AttnArgs &a, int n_seg, void *ws, size_t ws_bytes, cudaStream_t s);

}  // namespace csa2
