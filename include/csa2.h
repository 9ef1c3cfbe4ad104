/*
 * csa2.h -- C ABI of libcsa2, the CSA2 long-context attention step
 * (FP4 global KV cache, lightning indexer, top-k, sparse absorbed-query
 * attention with a sliding window) on one GB300 (sm_103a).
 *
 * Source pages cited below:
 *   [P1] "DeepSeek V4.1 Flash 아키텍처 분석" (plaidlabs.ai blog)
 *   [P2] "DeepSeek Multi-Head Latent Attention(MLA) 해부" (huny.dev blog)
 *   [P3] "DeepSeek V4.1 Flash 해부, KV 캐시는 줄고 사후학습 레시피는 그대로" (traillabs.ai)
 *   [P4] "매개변수는 커졌는데 메모리는 4분의 1, DeepSeek V4.1 Flash의 KV 캐시 다이어트" (ithotfix.com)
 *   [P5] "DeepSeek-V4: Towards Highly Efficient Million-Token Context Intelligence" (issue #58 translation)
 *
 * Conventions (all calls):
 *   - The caller owns every buffer.  Device pointers are CUDA device memory of
 *     the current device; host pointers are marked (host).  The library never
 *     allocates on these calls; scratch comes from a caller workspace whose
 *     size the matching *_workspace_size() returns.
 *   - Every device pointer must be 16-byte aligned (CSA2_ERR_ALIGN otherwise).
 *   - Calls are asynchronous on the given stream (a cudaStream_t; NULL = the
 *     legacy default stream).  They validate their arguments on the host first
 *     and return a status; they never abort and never throw.
 *   - Errors that only the device can see (an append beyond the capacity, an
 *     index outside the cache, a NaN score) set bits of the caller's int32
 *     *err_word (device memory, may be NULL to ignore) with atomicOr; the
 *     affected outputs are then unspecified.  Clear it before the calls and
 *     read it after synchronising.
 *   - csa2_last_error_detail() returns a thread-local text for the last
 *     non-OK status of this thread.
 */
#ifndef CSA2_H
#define CSA2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st *csa2_stream_t;

typedef enum csa2_status {
  CSA2_OK = 0,
  CSA2_ERR_NULL = 1,        /* a required pointer is NULL                       */
  CSA2_ERR_SHAPE = 2,       /* a size is outside its documented range           */
  CSA2_ERR_ALIGN = 3,       /* a device pointer is not 16-byte aligned          */
  CSA2_ERR_RANGE = 4,       /* an enum / k / ratio argument is out of range      */
  CSA2_ERR_UNSUPPORTED = 5, /* valid but not implemented (e.g. ratio-1 prefill) */
  CSA2_ERR_CUDA = 6,        /* a CUDA runtime call or kernel launch failed      */
  CSA2_ERR_WORKSPACE = 7    /* the workspace is NULL or smaller than required   */
} csa2_status;

/* bits of the device error word */
#define CSA2_DEVERR_CAPACITY 1u /* append past the cache capacity (nothing written) */
#define CSA2_DEVERR_INDEX 2u    /* an index / pool id outside the visible cache (skipped) */
#define CSA2_DEVERR_NAN 4u      /* a NaN index score (it ranks lowest)                */
#define CSA2_DEVERR_ROPE 8u     /* a position outside the RoPE table (nothing written) */
#define CSA2_DEVERR_TIMEOUT 16u /* a bounded device wait gave up (outputs unspecified)  */
#define CSA2_DEVERR_INEXACT 32u /* an index score may not be the exact dot (see csa2_index_score) */

/* sliding-window storage */
#define CSA2_SWA_BF16 0  /* 576 bf16 values, 1,152 B per token                         */
#define CSA2_SWA_MXFP8 1 /* 576 E4M3 codes + 18 E8M0 scales (one per 32), 594 B/token */

/* main-entry formats of the global cache (csa2_cache.entry_format):
 *   CSA2_ENTRY_FP4: V4.1, the 288 B record: lat_codes 256 B (E2M1 x 512),
 *     lat_scales 32 B (E4M3 per 16); RoPE sidecar rope_codes 32 B, rope_scales 4 B.
 *   CSA2_ENTRY_FP8: V4 ([P5] §2.3.4: FP8 for the entry except the RoPE dims,
 *     which stay BF16), for comparison: lat_codes 512 B (E4M3 x 512), lat_scales
 *     16 B (one E8M0 per 32 latent dims, e = floor(log2 amax) - 8, as the 8-bit
 *     window), rope_codes 128 B (the 64 rotated RoPE dims in bf16), rope_scales
 *     unused (may be NULL): 656 B.  The indexer key is MXFP4 (68 B) in both. */
#define CSA2_ENTRY_FP4 0
#define CSA2_ENTRY_FP8 1

/* input element types for csa2_kv_append */
#define CSA2_IN_F32 0
#define CSA2_IN_BF16 1

/* Fixed dimensions of the path (see the citations on csa2_cache). */
#define CSA2_D_LATENT 512 /* latent dims of a main-KV entry ([P1] "890 bytes/token")       */
#define CSA2_D_ROPE 64    /* decoupled RoPE dims ([P2] §3; [P5] §2.3.3 "last 64 dims")     */
#define CSA2_D_QK 576     /* score dims of an absorbed query: latent + RoPE ([P2] §4)      */
#define CSA2_D_INDEX 128  /* indexer head dim c_I ([P5] §4.2.1)                            */
#define CSA2_D_CMP 704    /* one compression row: 576 main dims then 128 indexer dims      */
#define CSA2_WINDOW 128   /* sliding window n_win ([P5] §4.2.1)                            */
#define CSA2_MAX_TOPK 2048
#define CSA2_MAX_HEADS 128

/*
 * One global-KV cache (the output of one Full layer; Reindex and Reuse layers
 * read it).  Every plane is [batch][capacity][bytes], sequence-major, so one
 * sequence's entries are contiguous.  Per entry ([P1] "890 bytes/token";
 * [P4] "890이 맞아떨어지는 계산"):
 *   lat_codes   256 B  E2M1 codes of the 512 latent dims, byte j = code(2j) | code(2j+1) << 4
 *   lat_scales   32 B  one E4M3 scale per 16 dims                 -> 288 B main entry
 *   rope_codes   32 B  E2M1 codes of the 64 rotated RoPE dims (sidecar of the MLA split, [P2] §3)
 *   rope_scales   4 B  one E4M3 scale per 16                       -> 36 B sidecar
 *   idx_codes    64 B  E2M1 codes of the 128-dim indexer key
 *   idx_scales    4 B  one E8M0 scale per 32 (MXFP4)               -> 68 B indexer entry
 *   The two indexer planes are tile-major: [batch][ceil(capacity/128)][8192 B]
 *   and [batch][ceil(capacity/128)][512 B], in the operand layout of the
 *   block-scaled tensor-core MMA.  For entry e (tile = e/128, m = e%128) the
 *   16 code bytes of 32-value block j sit at tile*8192 + j*2048 + m*16 and its
 *   scale byte at tile*512 + 16*(m%32) + 4*(m/32) + j.  csa2_cache_plane_bytes()
 *   gives every plane's size.
 * swa_codes / swa_scales: the sliding-window ring, [batch][128][576] codes
 *   (E4M3 bytes, or bf16 when swa_dtype == CSA2_SWA_BF16) and [batch][128][32]
 *   scale bytes (18 used, MXFP8 only); token t lives in slot t % 128 ([P5]
 *   §3.5.1: the window is a fixed-size per-sequence state).
 * cmp_buf: ratio 2 only, float [batch][4][4][704]: the last tokens' compression
 *   rows (C^a, C^b, Z^a, Z^b) at slot t % 4, carried between appends ([P5] §3.5.1
 *   "Compression Buffer").
 * n_tokens: int64 [batch] tokens appended so far (device; csa2_kv_append and
 *   csa2_prefill_chunk advance it).  A ratio-r cache holds floor(n_tokens/r) entries.
 * ratio: 1 (one token per entry, decoder) or 2 (two tokens per entry, encoder;
 *   [P1] "Global KV는 네 곳에서 만든다", [P4] 178 B per token).
 *
 * Paged layout ([P5] §3.5.1 "Sparse Attention Kernel Co-Design": the global
 * entries live in fixed-size blocks whose token count is a multiple of the
 * compression ratios; the window and the compression buffer are
 * per-sequence state, "State Cache"): with block_table != NULL the six entry
 * planes hold n_pages physical pages of page_entries entries each, page-major
 * (lat_codes [n_pages][page_entries][256], ..., the indexer planes
 * [n_pages][page_entries/128][8192 B] and [..][512 B] in the same tile layout),
 * and entry e of sequence b is entry e % page_entries of physical page
 * block_table[b * max_pages + e / page_entries].  page_entries is a multiple of
 * 128 (an indexer tile never straddles pages; a page's tokens are then a
 * multiple of every ratio and of the 8-position pool block), capacity must
 * equal max_pages * page_entries, and page ids lie in 0..n_pages-1 (an id
 * outside raises the INDEX device bit and the access is skipped).  Pages may be
 * shared between sequences only for entries they hold in common; the caller
 * fills the table before the entries are appended.  The window ring, the
 * compression buffer and n_tokens stay indexed by sequence.  block_table ==
 * NULL: the dense layout above (page fields ignored).
 */
typedef struct csa2_cache {
  int32_t batch;
  int32_t capacity; /* entries per sequence */
  int32_t ratio;
  int32_t swa_dtype;
  uint8_t *lat_codes, *lat_scales;
  uint8_t *rope_codes, *rope_scales;
  uint8_t *idx_codes, *idx_scales;
  uint8_t *swa_codes, *swa_scales;
  float *cmp_buf;
  int64_t *n_tokens;
  const int32_t *block_table; /* [batch][max_pages] physical page ids, or NULL (dense) */
  int32_t page_entries;       /* entries per page: a multiple of 128 */
  int32_t max_pages;          /* pages a sequence may use: capacity / page_entries */
  int32_t n_pages;            /* physical pages in the entry planes */
  int32_t entry_format;       /* CSA2_ENTRY_FP4 (V4.1) or CSA2_ENTRY_FP8 (V4) */
} csa2_cache;

/* Ratio-2 compression inputs ([P5] §2.3.1 "압축된 Key-Value Entry"): per token
 * rows of C^a, C^b, Z^a, Z^b ([batch][n_new][704], device fp32) and the
 * positional biases B^a, B^b ([2][704], device fp32). */
typedef struct csa2_compress_in {
  const float *ca, *cb, *za, *zb;
  const float *ba, *bb;
} csa2_compress_in;

/* Bytes each plane of a cache needs (host helper; no device work). */
size_t csa2_cache_plane_bytes(int32_t batch, int32_t capacity, int32_t plane /* 0..9 as listed */,
                              int32_t swa_dtype);
/* Bytes of entry plane 0..5 in the paged layout (n_pages pages of page_entries). */
size_t csa2_paged_plane_bytes(int32_t n_pages, int32_t page_entries, int32_t plane);
/* Bytes one entry takes in plane 0..5 for an entry format (0 for an unknown
 * format or plane; the dense and paged plane sizes above are for
 * CSA2_ENTRY_FP4, scale them by this for CSA2_ENTRY_FP8). */
size_t csa2_entry_plane_bytes(int32_t entry_format, int32_t plane);

/*
 * csa2_rope_table (host): cos/sin table for the 64 RoPE dims, rope_cs[pos][i][2]
 * = (cos, sin)(pos * theta^(-2i/64)) for i < 32, evaluated in double and rounded
 * to fp32, positions 0..n_pos-1 ([P5] §2.3.3 "Partial Rotary Positional
 * Embedding"; pairs (2i, 2i+1) interleaved).  out_host holds n_pos*64 floats.
 */
csa2_status csa2_rope_table(double theta, int64_t n_pos, float *out_host);

/*
 * csa2_kv_append: quantise n_new new tokens of every sequence into the cache,
 * at positions n_tokens[b] .. n_tokens[b]+n_new-1, then advance n_tokens.
 *   ratio 1: kv [batch][n_new][576] (512 latent, 64 RoPE dims not yet rotated),
 *            idx_key [batch][n_new][128], element type in_dtype; cmp = NULL.
 *            Entry t = token t: RoPE at position t, then quantise ([P4]
 *            "890이 맞아떨어지는 계산": quantisation after RoPE).
 *   ratio 2: cmp != NULL, kv = idx_key = NULL.  Entry i is emitted when tokens
 *            2i, 2i+1 are present: per channel a softmax over the 4 rows
 *            [Z^a_2i + B^a_0, Z^a_2i+1 + B^a_1, Z^b_2i-2 + B^b_0, Z^b_2i-1 + B^b_1]
 *            and the gated sum of the matching C rows ([P5] §2.3.1), computed in
 *            fp64 and rounded to fp32, then RoPE at position 2i, then quantised.
 *            Rows of earlier appends come from cmp_buf.
 *   Window: each of the last min(n_new, 128) tokens fills slot t % 128 with its
 *            own vector (ratio 1: kv; ratio 2: C^a[0:576]) rotated at t, in 8 bits
 *            or bf16 ([P1] "890 bytes/token": the window KV stays in FP8).
 * rope_cs: device table from csa2_rope_table with rope_len positions.
 * cmp_dbg: NULL, or device fp32 [batch][n_new/2+1][704] receiving each emitted
 *   ratio-2 entry before RoPE (row e = the e-th entry emitted by this call).
 * Device errors: CAPACITY (a sequence would exceed capacity; nothing written
 *   for it), ROPE (a position >= rope_len).
 */
csa2_status csa2_kv_append(const csa2_cache *cache, const void *kv, const void *idx_key,
                           int32_t in_dtype, const csa2_compress_in *cmp, const float *rope_cs,
                           int64_t rope_len, int32_t n_new, float *cmp_dbg, int32_t *err_word,
                           csa2_stream_t stream);

/*
 * csa2_index_score: lightning-indexer scores ([P5] §2.3.1, "I_{t,s} = sum_h
 * w_{t,h} ReLU(q_{t,h} . K_s)"), with the query quantised to MXFP4 like the
 * keys (the indexer QK product runs in FP4, [P5] §2.3.4).
 *   q_idx: bf16 [batch][n_heads_idx][128]; w: fp32 [batch][n_heads_idx];
 *   q_pos: int64 [batch] query positions; entry s is visible iff
 *          s < floor(q_pos / ratio) ([P5] §2.3.1).
 *   d_h is the dot of the dequantised vectors, rounded once to fp32.  That holds
 *   when the block exponents e_q,j + e_k,j of a (head, key) pair span at most 9
 *   binades over the blocks whose two scale codes are nonzero (always the case
 *   for N(0,1)-like data); a visible key whose pair with some head spans more
 *   raises the INEXACT bit (its scores are then unspecified in the last bits);
 *   score = fma chain over heads in order: acc = fma(w_h, max(d_h, +0), acc).
 * FULL (pool == NULL): scores[b][s] for every visible s (others untouched).
 * POOL (Reindex, [P1] "512개를 고르기 위해 ..."): pool [batch][pool_blocks] int32
 *   ascending block ids (-1 = empty); scores[b][j*pool_block_size + i] is the
 *   score of position pool[b][j]*pool_block_size + i when it is visible.
 * score_stride: floats per sequence in scores (>= capacity for FULL,
 *   >= pool_blocks*pool_block_size for POOL).  n_heads_idx in 1..128.
 * score_aux: NULL, or a device buffer of csa2_score_aux_size(batch,
 *   score_stride) bytes that receives a sideband for csa2_topk: per row a
 *   histogram of the scores' top 13 order bits and, in FULL mode, the max of
 *   every 8-position block with its histogram.  Owned by the caller; valid
 *   until the scores change.  Building it here costs no extra pass over them.
 * ws: device workspace of csa2_index_score_workspace_size() bytes (the
 *   quantised queries in the tensor-core operand layout).
 * The contraction runs on the tensor cores (block-scaled MXFP4 MMA) for FULL
 * and for POOL with pool_block_size 8; other block sizes use CUDA cores (the
 * sideband is then built by a second kernel over the scores).
 */
size_t csa2_index_score_workspace_size(int32_t batch, int32_t n_heads_idx);
size_t csa2_score_aux_size(int32_t batch, int64_t score_stride);
csa2_status csa2_index_score(const csa2_cache *cache, const uint16_t *q_idx, const float *w,
                             int32_t n_heads_idx, const int64_t *q_pos, const int32_t *pool,
                             int32_t pool_blocks, int32_t pool_block_size, float *scores,
                             int64_t score_stride, void *score_aux, void *ws, size_t ws_bytes,
                             int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_topk: top-k selector ([P5] §2.3.1 "Top-k(I_{t,:})") over the candidates
 * csa2_index_score scored (same ratio / q_pos / pool arguments), ordered by
 * score descending then position ascending (ties go to the lower position;
 * -0 == +0; NaN ranks lowest and raises the NAN bit).  idx_out [batch][k]
 * receives the chosen positions in ascending order, padded with -1.
 * k in 1..2048.
 * score_aux: the sideband csa2_index_score wrote for these scores, or NULL
 *   (it is then rebuilt from the scores inside ws, one more pass over them).
 * FULL mode only: when pool_out != NULL also builds the candidate pool of the
 * Hierarchical Sparse Indexer ([P1], [P4]): positions are grouped in aligned
 * blocks of pool_block_size = 8, a block's score is the max over its visible
 * positions, and the top out_pool_blocks (1..2048) blocks by (max desc, block
 * asc) are written ascending to pool_out [batch][out_pool_blocks] (padded with
 * -1), with their number in pool_count [batch].
 * ws: device workspace of csa2_topk_workspace_size() bytes (enough with or
 *   without score_aux).
 * The selection is exact for any input; rows whose k-th score falls in a bin
 * holding more than 4096 scores take a slower exact path.
 */
size_t csa2_topk_workspace_size(int32_t batch, int64_t score_stride, int32_t k,
                                int32_t out_pool_blocks);
csa2_status csa2_topk(const float *scores, int64_t score_stride, const void *score_aux,
                      int32_t batch, int32_t ratio, const int64_t *q_pos, const int32_t *pool,
                      int32_t pool_blocks, int32_t pool_block_size, int32_t k, int32_t *idx_out,
                      int32_t out_pool_blocks, int32_t *pool_out, int32_t *pool_count, void *ws,
                      size_t ws_bytes, int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_topk_noalloc: csa2_topk without a caller workspace, for callers that
 * may not allocate device memory while they run (a host framework that owns all
 * device allocations, a service whose memory budget is fixed at start-up, code
 * that must not hit the allocator's implicit synchronisation).  The source pages
 * have no counterpart: this is a library convenience, not a step of the method.
 * Same arguments and results as csa2_topk minus score_aux, ws and ws_bytes (the
 * sideband is always rebuilt from the scores).  Its scratch is a 4 MiB array
 * compiled into the library, resident on every GPU that loads it until the
 * process exits; calls needing more (csa2_topk_workspace_size() > 4 MiB, i.e.
 * large batch x score_stride) return CSA2_ERR_WORKSPACE with the sizes in
 * csa2_last_error_detail().  The first call on each device looks up the
 * array's device address (a runtime query), so make that first call before any
 * stream capture; the address is kept for the process, so a cudaDeviceReset
 * after that first call is not supported.  Every call shares the array and leaves its contents behind
 * (each call clears and rewrites what it reads): calls whose kernels may
 * overlap on the GPU -- different streams without ordering -- race.
 */
csa2_status csa2_topk_noalloc(const float *scores, int64_t score_stride, int32_t batch, int32_t ratio,
                              const int64_t *q_pos, const int32_t *pool, int32_t pool_blocks,
                              int32_t pool_block_size, int32_t k, int32_t *idx_out,
                              int32_t out_pool_blocks, int32_t *pool_out, int32_t *pool_count,
                              int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_mask_to_pool: the Reindex selection in the form of the published
 * reference code ([P1] "DeepSeek V4.1 Flash 아키텍처 분석", §"공개 코드를 읽어 보니
 * 남는 차이": Indexer.forward scores every key, then masks the positions outside
 * the candidates), kept for comparison with scoring only inside the pool.
 * scores [batch][score_stride] FULL-mode scores (csa2_index_score with pool ==
 * NULL); every visible position s < floor(q_pos[b] / ratio) whose block
 * s / pool_block_size is not among pool[b] (ascending block ids, -1 padded,
 * pool_blocks per row) is set to -inf in place.  csa2_topk (FULL, k) over the
 * masked row then selects what csa2_topk over the pool's scores selects
 * whenever the pool holds at least k visible positions.  pool_block_size 1..64.
 */
csa2_status csa2_mask_to_pool(float *scores, int64_t score_stride, int32_t batch, int32_t ratio,
                              const int64_t *q_pos, const int32_t *pool, int32_t pool_blocks,
                              int32_t pool_block_size, csa2_stream_t stream);

/*
 * csa2_sparse_attn_decode: core attention of one decode step over the k
 * selected entries and the window ([P5] §2.3.1 "Shared Key-Value MQA": each
 * entry is key and value; [P2] §4 absorbed query: logits over 576 dims, values
 * the 512 latent dims; [P5] §2.3.3 window branch and attention sink).
 *   q: bf16 [batch][n_heads][576] (latent 512 then rotated RoPE 64);
 *   idx: int32 [batch][k] positions (-1 = empty) -- a Reuse layer passes its
 *        leader's list and cache ([P3] "CSA2의 세 가지 모드");
 *   window: tokens max(0, q_pos-127) .. q_pos that are < n_tokens[b];
 *   sink: fp32 [n_heads] or NULL; sm_scale: logit scale.
 *   z_j = sm_scale * q . e_j; p_j = exp(z_j - M) / (sum_j exp(z_j - M) + exp(sink_h - M));
 *   out: fp32 [batch][n_heads][512] = sum_j p_j c_j; lse: fp32 [batch][n_heads]
 *   = M + log(denominator) (-inf when there is nothing to attend to).
 * n_heads: a multiple of 16, 16..128.  k: 1..2048.
 * Batch invariance ([P5] §3.3): a row's result is bit-identical whatever the
 *   batch it is computed in.  Its 32-entry chunks (the k selected entries, then
 *   the window) are dealt to S = min(4, chunks) segments, S a function of k
 *   alone; each segment runs its own online softmax and the row merges the S
 *   partials in segment order.  Only the launch shape follows the batch and
 *   the GPU's SM count: how many CTAs share a row's segments, and how many
 *   heads (64, 32 or 16) a CTA takes.
 * ws: device workspace of csa2_attn_workspace_size() bytes, 16-byte aligned:
 *   the partial (O, m, l) of each segment of a row (S x 131 KB per row and
 *   64 heads), written and read within the call; calls that may run
 *   concurrently need separate workspaces.
 * Device errors: INDEX (an index >= the visible entries; that entry is skipped).
 */
size_t csa2_attn_workspace_size(int32_t batch, int32_t n_heads, int32_t k);
csa2_status csa2_sparse_attn_decode(const csa2_cache *cache, const uint16_t *q, int32_t n_heads,
                                    const int64_t *q_pos, const int32_t *idx, int32_t k,
                                    const float *sink, float sm_scale, float *out, float *lse,
                                    void *ws, size_t ws_bytes, int32_t *err_word,
                                    csa2_stream_t stream);

/*
 * csa2_prefill_chunk: encoder-style chunked prefill of sequence `seq` of a
 * ratio-2 cache.  Appends the Q tokens (as csa2_kv_append, ratio 2), then for
 * every query i (position P+i, P = n_tokens[seq] before the call): scores all
 * visible entries s < floor((P+i)/2) with its own indexer query (a dense FP4
 * contraction), keeps its top k, and attends over them plus its window tokens
 * max(0, P+i-127) .. P+i ([P5] §2.3.1, §2.3.3).
 *   cmp: rows [Q][704] for this sequence; q_idx bf16 [Q][n_heads_idx][128];
 *   w fp32 [Q][n_heads_idx]; q bf16 [Q][n_heads][576];
 *   idx_out int32 [Q][k]; out fp32 [Q][n_heads][512]; lse fp32 [Q][n_heads].
 * ws: device workspace of csa2_prefill_workspace_size() bytes (queries are
 *   scored, selected and attended in blocks: the block holds ~256 MB of fp32
 *   score rows, rounded down to a multiple of twice the current device's SM
 *   count, so the size depends on the device the call runs on; query it with
 *   that device current).
 * Each query's attention is one pass over its entries (one segment), so its
 * bits do not depend on the chunk's size either; they may differ in the last
 * bits from a decode step at the same position (csa2_sparse_attn_decode merges
 * S segments), within the attention tolerance.
 * Ratio-1 caches return CSA2_ERR_UNSUPPORTED.
 */
size_t csa2_prefill_workspace_size(int32_t Q, int32_t capacity, int32_t n_heads_idx,
                                   int32_t n_heads, int32_t k);
csa2_status csa2_prefill_chunk(const csa2_cache *cache, int32_t seq, const csa2_compress_in *cmp,
                               const float *rope_cs, int64_t rope_len, int32_t Q,
                               const uint16_t *q_idx, const float *w, int32_t n_heads_idx,
                               const uint16_t *q, int32_t n_heads, int32_t k, const float *sink,
                               float sm_scale, int32_t *idx_out, float *out, float *lse, void *ws,
                               size_t ws_bytes, int32_t *err_word, csa2_stream_t stream);

/*
 * Ragged calls: a batch whose sequences bring different numbers of new tokens
 * (chunks of prompts beside single decoded tokens).  The tokens are packed one
 * sequence after the other: sequence b has rows cu[b] .. cu[b+1]-1 of every
 * per-token array, cu int32 [batch+1] in device memory with cu[0] = 0,
 * non-decreasing; a sequence may have none.  total is the number of rows the
 * arrays hold (host): rows from cu[batch] on belong to no sequence, so one call
 * (or captured graph) may serve batches that fill it differently; outputs of
 * those rows are left as they were.  max_new is the caller's bound on
 * cu[b+1]-cu[b] (host; it decides launch shapes): a sequence that breaks it, or
 * whose cu does not fit the arrays, is skipped with the INDEX bit, and so is one
 * whose rows a list that decreases somewhere gives to another one too.
 *
 * Window rows of a chunk.  The ring holds a sequence's last 128 tokens, but a
 * chunk's earlier queries look further back: for them the append leaves, per
 * sequence, the 128 tokens before the chunk followed by the chunk's own, in the
 * window's format, rows cu[b] + 128 b .. : row cu[b] + 128 b + i is token
 * P - 128 + i, P = n_tokens[b] before the append (zeros where that is
 * negative).  win_codes: (total + 128 batch) rows of 576 (MXFP8) or 1,152
 * (bf16) bytes; win_scales: as many rows of 32 bytes (MXFP8; may be NULL for
 * bf16).  csa2_chunk_window_bytes() gives the two sizes (plane 0, 1).
 */
size_t csa2_chunk_window_bytes(int32_t batch, int32_t total, int32_t swa_dtype, int32_t plane);

/*
 * csa2_kv_append_ragged: csa2_kv_append for a ragged batch; the records, the
 * ring, the compression buffer and n_tokens end up as if every sequence had
 * been appended by itself.
 *   ratio 1: kv rows of 576, idx_key rows of 128, element type in_dtype, row t at
 *            kv + t * kv_stride elements (kv_stride >= 576, key_stride >= 128, both
 *            multiples of 8: a row may be a slice of a wider projection);
 *            cmp = NULL.
 *   ratio 2: cmp rows [total][704] each; kv = idx_key = NULL, strides ignored.
 *   win_codes / win_scales: the chunk's window rows (above), or NULL.
 * The call reads the ring before it overwrites it; win_codes must not be in use
 * by an earlier call on another stream.  total 0 and max_new 0 are valid calls
 * (nothing done), here and in csa2_chunk_attn.
 * Device errors: CAPACITY, ROPE (nothing written for the sequence, its n_tokens
 * stays), INDEX (a page id outside the pool, cu, max_new).
 */
csa2_status csa2_kv_append_ragged(const csa2_cache *cache, const void *kv, int64_t kv_stride, const void *idx_key,
                                  int64_t key_stride, int32_t in_dtype, const csa2_compress_in *cmp,
                                  const int32_t *cu_new, int32_t total, int32_t max_new, const float *rope_cs,
                                  int64_t rope_len, uint8_t *win_codes, uint8_t *win_scales, int32_t *err_word,
                                  csa2_stream_t stream);

/* element types of what the reads and the chunk attention write */
#define CSA2_OUT_F32 0
#define CSA2_OUT_BF16 1

/*
 * csa2_kv_read: cached entries back as the values they stand for.
 *   Rows cu_rows[b] .. cu_rows[b+1]-1 read sequence b: row r is entry
 *   pos[r] (int32 [total]; any order, repeats allowed, negative = an empty row)
 *   when pos != NULL, else entry start[b] + (r - cu_rows[b]) (int64 [batch]).
 *   out_main: rows of 576 (512 latent, then the 64 rotated RoPE dims), or NULL;
 *   out_key: rows of 128 (the indexer key), or NULL; out_dtype, row strides in
 *   elements (>= 576 / 128, multiples of 8).  Every value is exact in fp32, and in
 *   bf16 too for FP4 records and keys, bf16 RoPE dims, and MXFP8 latents down to
 *   bf16's step of 2^-133, to which smaller ones are rounded.
 *   Empty rows are zeros.  Rows of no sequence, or of a skipped one, are left as
 *   they were.
 * Device errors: INDEX (an entry not in the cache, floor(n_tokens/ratio) or more,
 * a negative start, or a bad page id: the row is zeros; cu).
 */
csa2_status csa2_kv_read(const csa2_cache *cache, const int32_t *cu_rows, int32_t total, const int32_t *pos,
                         const int64_t *start, void *out_main, int64_t main_stride, void *out_key, int64_t key_stride,
                         int32_t out_dtype, int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_window_read: the sliding window's tokens in order, out [batch][128][576]
 * of out_dtype: row i is token n_tokens[b] - 128 + i (zeros where negative).
 */
csa2_status csa2_window_read(const csa2_cache *cache, void *out, int32_t out_dtype, csa2_stream_t stream);

/*
 * csa2_chunk_attn: dense attention of a ragged batch's new tokens (already
 * appended) over every visible entry of the cache and the window: the layer
 * form without a selection ([P5] §2.3.2 dense attention over compressed
 * entries; window-only layers; contexts no longer than the top-k).  Definition
 * and operands as csa2_sparse_attn_decode with every visible entry selected.
 *   q: bf16 [total][n_heads][576]; query row cu_q[b] + i of a sequence with n
 *      new tokens is at position p = n_tokens[b] - n + i; it sees entries
 *      s < floor(p / ratio) and window tokens max(0, p-127) .. p.
 *   win_codes / win_scales: the append's window rows for the same cu, or NULL:
 *      the window then comes from the ring, which holds what single new tokens
 *      need (a query whose window reaches behind the ring raises INDEX and goes
 *      without those tokens).
 *   sink: fp32 [n_heads] or NULL; sm_scale finite.
 *   out: out_dtype [total][n_heads][512]; lse: fp32 [total][n_heads].
 *   A row that sees nothing (bad pages, no sink) is zeros with lse -inf.  Values
 *   of tokens that a row does not see never reach it: a window token with an
 *   infinite or NaN latent (a bf16 window holds them as they are) makes the rows
 *   that see it NaN, and only those, as does a V4 entry with a NaN among its RoPE
 *   dims.  Other records hold no NaN: the appends write none.
 *   Precision: sums, softmax statistics and out before its rounding in fp32, FP4
 *   records exact.  An element of out is off by at most about
 *   sum_j p_j (2^-11 |c_j| + 2^-25 s_j) + 2^-29 W sum_j |c_j| / s_j with
 *   W = max_j p_j s_j: the weights, and the values of V4 entries and of the window,
 *   are fp16 in the products.  s_j is 1 for FP4 records and for keys whose largest
 *   magnitude (RoPE dims included) lies in 2^0 .. 2^16, else 2^(e-8) for one of
 *   2^e .. 2^(e+1), 2^-24 at least.  So a value below 2^-25 of its key's largest
 *   magnitude may be lost, and so may keys with a largest magnitude below about
 *   2^-20 beside much larger ones, or below 2^-49.
 * n_heads: a multiple of 16, 16..128.  The work is split over the GPU by the
 * batch's total work, so a row's last bits may change with the batch (use
 * csa2_sparse_attn_decode where batch invariance is needed); equal calls give
 * equal bits.
 * ws: device workspace of csa2_chunk_attn_workspace_size() bytes (for the
 * current device); calls that may overlap need one each.
 * Device errors: INDEX (a page id outside the pool: those entries are skipped;
 * cu, max_new; a window behind the ring), TIMEOUT.
 */
size_t csa2_chunk_attn_workspace_size(int32_t batch, int32_t total, int32_t n_heads);
csa2_status csa2_chunk_attn(const csa2_cache *cache, const uint16_t *q, int32_t n_heads, const int32_t *cu_q,
                            int32_t total, int32_t max_new, const uint8_t *win_codes, const uint8_t *win_scales,
                            const float *sink, float sm_scale, void *out, int32_t out_dtype, float *lse, void *ws,
                            size_t ws_bytes, int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_pages_resize: the pages of a paged cache for the lengths its sequences are
 * to have ([P5] §3.5.1), without the host.  Sequence b is to hold
 *   need_b = ceil(floor(n_b / ratio) / page_entries) pages,
 *   n_b = target[b] (int64 [batch]), or, when target is NULL, n_tokens[b] plus the
 *   new tokens cu_new gives it (cu_new NULL: none; cu_new, total, max_new as in the
 *   ragged calls, before the append).
 * pool: held int32 [batch], the pages each sequence holds (entries 0..held-1 of its
 *   block_table row); free int32 [n_pages], a stack of free page ids, n_free int32
 *   [1] of them.  All device memory that the caller owns, as is block_table, which
 *   this call writes.  A page is in one place: on the stack or in one sequence's row.
 * Pages beyond need go back to the stack and their entries become -1 (a sequence
 *   that ended: length 0; drafted tokens that were refused: the shorter length).
 *   With R of them, the j-th in sequence and page order goes to
 *   free[n_free + R - 1 - j].  Then the sequences that need more take pages from the
 *   top, in order: the k-th page is the one at free[n_free + R - 1 - k].  A sequence
 *   gets all it needs or nothing: from the first whose need does not fit on, no
 *   sequence that needs more gets any.  Pages are handed out, not cleared.
 * granted: int32 [batch] or NULL, 1 where a sequence holds what it needs, else 0.
 * Equal calls give equal tables; taking pages and giving them back restores both.
 * Device errors, the sequence left as it was: CAPACITY (need_b > max_pages), INDEX
 *   (cu_new, max_new, a negative length, held outside 0..max_pages, an id outside the
 *   pool among the pages that would go back).  INDEX with nothing done: n_free outside
 *   0..n_pages, or more pages than the pool has.  A pool that runs out is no error: see
 *   granted.
 */
typedef struct csa2_page_pool {
  int32_t *free;   /* [n_pages] */
  int32_t *n_free; /* [1] */
  int32_t *held;   /* [batch] */
} csa2_page_pool;
csa2_status csa2_pages_resize(const csa2_cache *cache, const csa2_page_pool *pool, const int64_t *target,
                              const int32_t *cu_new, int32_t total, int32_t max_new, int32_t *granted, int32_t *err_word,
                              csa2_stream_t stream);

/*
 * csa2_slot_map: position and place of every new token of a ragged batch, before
 * they are appended (cu_new, total, max_new as there).
 *   pos: int64 [total] or NULL, n_tokens[b] + i for row cu_new[b] + i, as
 *        csa2_query_latent takes it; slots: int64 [total] or NULL, the physical
 *        entry (page * page_entries + offset, or b * capacity + entry in a dense
 *        cache) of the token's entry, for planes of the caller's own beside the
 *        cache's; -1 when the entry is not complete after this call (ratio 2).
 * Rows of no sequence, or of a skipped one, get -1 in both.
 * Device errors: INDEX (cu_new, max_new; a page id outside the pool: slot -1; a
 * negative n_tokens), CAPACITY (an entry behind the capacity: slot -1).
 */
csa2_status csa2_slot_map(const csa2_cache *cache, const int32_t *cu_new, int32_t total, int32_t max_new, int64_t *slots,
                          int64_t *pos, int32_t *err_word, csa2_stream_t stream);

/*
 * 4-bit block-scaled matrices: the formats the cache is held in, for the layer's
 * own projections (their weights, and the activations they multiply).
 *   CSA2_FP4_NV: E2M1 codes, one E4M3 scale per 16 columns (as the main entry) and
 *     one power of two r per row.  r is the least one, 2^-62 at least, with
 *     largest magnitude of the row / r <= 2688 = 448 x 6; then per group
 *     s = E4M3(amax / (6 r)), codes E2M1(x / (r s)) (x's sign bit, of a zero too),
 *     zeros where s is 0.
 *   CSA2_FP4_MX: E2M1 codes, one E8M0 scale per 32 columns (as the indexer key);
 *     r = 1.
 *   Value: code x scale x r.  A row that holds an infinity or NaN (NV: also one whose
 *   largest magnitude is above 2688 x 2^62) gets r = NaN and raises the NAN bit: what
 *   is read or computed from it is NaN.
 * Planes (csa2_fp4_plane_bytes, plane 0 and 1):
 *   tiles       records of 128 rows x 128 columns, row tile by row tile, in the operand
 *               layout of the block-scaled tensor-core MMA: 8,192 B of codes, the 16
 *               bytes of 32-column piece j of row m at j * 2048 + m * 16, then the scales,
 *               NV (1,024 B): (g / 4) * 512 + 16 (m % 32) + 4 (m / 32) + g % 4, group g of
 *               8; MX (512 B): 16 (m % 32) + 4 (m / 32) + j
 *   row_scales  float r per row
 * Rows behind `rows` in the last tile are not written, and what they hold does not matter.
 * rows 0..2^24, cols 1..2^17.
 */
#define CSA2_FP4_NV 0
#define CSA2_FP4_MX 1
typedef struct csa2_fp4_matrix {
  int32_t rows, cols;
  int32_t format;
  uint8_t *tiles;
  float *row_scales;
} csa2_fp4_matrix;
size_t csa2_fp4_plane_bytes(int32_t rows, int32_t cols, int32_t format, int32_t plane);

/*
 * csa2_fp4_quant: the rows x, fp32 or bf16 (in_dtype, CSA2_IN_*), row t at
 * x + t * x_stride elements (x_stride >= cols, a multiple of 8), into the matrix m.
 * csa2_fp4_read: the values m stands for, out_dtype (CSA2_OUT_*), rows out_stride
 * elements apart (>= cols, a multiple of 8); exact in fp32, and in bf16 too.
 * x or out must not overlap m's planes.  Device errors (quant): NAN, TIMEOUT.
 */
csa2_status csa2_fp4_quant(const csa2_fp4_matrix *m, const void *x, int64_t x_stride, int32_t in_dtype, int32_t *err_word,
                           csa2_stream_t stream);
csa2_status csa2_fp4_read(const csa2_fp4_matrix *m, void *out, int64_t out_stride, int32_t out_dtype, csa2_stream_t stream);

/*
 * csa2_fp4_product: out[m][n] = sum_k x[m][k] w[n][k], x and w of one format and
 * as many columns, out_dtype [x->rows] rows of w->rows values out_stride elements
 * apart (>= w->rows, a multiple of 8).  Products and block scales are exact, sums in
 * fp32 (in an order that the sizes decide; equal calls give equal bits), the rows'
 * powers of two applied to the sum, then rounded to out_dtype.  A row's last bits may
 * change with the number of rows.  out must not overlap x or w.
 * Device errors: TIMEOUT.
 */
csa2_status csa2_fp4_product(const csa2_fp4_matrix *x, const csa2_fp4_matrix *w, void *out, int64_t out_stride,
                             int32_t out_dtype, int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_query_latent: a layer's queries into the latent space, the absorbed form that
 * the attention calls take ([P2] §4: q W^UK), with the RoPE dims rotated as the
 * appends rotate the keys'.  Per row t and head h
 *   out[t][h][0:512]   = sum_k q[t][h][k] w_uk[h][k][0:512], k < dim
 *   out[t][h][512:576] = q[t][h][dim:dim+64] rotated at position pos[t]
 *   q: bf16, row t at q + t * q_stride elements, its heads dim + 64 values each one
 *      after the other (q_stride >= n_heads (dim + 64), a multiple of 8);
 *   w_uk: bf16, head h's dim rows of 512 at w_uk + h * w_stride (>= dim x 512, a
 *      multiple of 8: keys' and values' rows may lie together);
 *   pos: int64 [total], as csa2_slot_map leaves them; out: bf16 [total][n_heads][576].
 * Rows with a negative position are left as they were.  Sums in fp32, rounded once.
 * n_heads 1..128, dim a multiple of 16, 16..128.
 * Device errors: ROPE (a position >= rope_len: the row is left as it was), TIMEOUT.
 */
csa2_status csa2_query_latent(const uint16_t *q, int64_t q_stride, int32_t total, int32_t n_heads, int32_t dim,
                              const uint16_t *w_uk, int64_t w_stride, const int64_t *pos, const float *rope_cs,
                              int64_t rope_len, uint16_t *out, int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_value_project: attended latent rows to the heads' values ([P2] §4: the
 * deferred W^UV).  Per row t and head h
 *   out[t][h dim + j] = sum_c o[t][h][c] w_uv[h][j][c], c < 512, j < dim
 *   o: fp32 or bf16 (in_dtype, CSA2_IN_*), row t at o + t * o_stride elements, its
 *      heads 512 values each (o_stride >= n_heads x 512, a multiple of 8);
 *   w_uv: bf16, head h's dim rows of 512 at w_uv + h * w_stride, as w_uk;
 *   out: bf16, row t at out + t * out_stride (>= n_heads x dim, a multiple of 8).
 * Sums in fp32, rounded once; fp32 rows enter as three bf16 parts that add up to them
 * (but for bits below 2^-126; an infinite weight may give NaN, 0 being among the parts).
 * n_heads 1..128, dim a multiple of 16, 16..128.  Device errors: TIMEOUT.
 * In both calls a row's last bits may change with the number of rows; equal calls
 * give equal bits; out must not overlap what is read.
 */
csa2_status csa2_value_project(const void *o, int64_t o_stride, int32_t in_dtype, int32_t total, int32_t n_heads, int32_t dim,
                               const uint16_t *w_uv, int64_t w_stride, uint16_t *out, int64_t out_stride, int32_t *err_word,
                               csa2_stream_t stream);

/*
 * csa2_mxf4_peak_launch: measurement helper (not a step of the method).
 * Launches n_ctas CTAs that each issue `iters` back-to-back block-scaled FP4
 * tensor-core MMAs (tcgen05 kind::mxf4, M 128 x N 128 x K 64, the index score's
 * instruction) on operands resident in shared memory: n_ctas x iters x
 * 2,097,152 FLOP.  The caller times it (events on `stream`) to get the dense
 * FP4 rate the prefill indexer's tensor-pipe utilisation is reported against
 * ([P5] §2.3.4: the indexer QK product runs in FP4).  sink: NULL, or device
 * uint32 [n_ctas] receiving one accumulator word per CTA.  err_word: the
 * TIMEOUT bit if the final wait gave up.  n_ctas 1..4096, iters 2..2^24.
 */
csa2_status csa2_mxf4_peak_launch(int32_t n_ctas, int32_t iters, uint32_t *sink, int32_t *err_word,
                                  csa2_stream_t stream);

/*
 * csa2_bounded_wait_check: self-check of the failure path (not a step of the
 * method).  Every wait inside the library's kernels is bounded: a wait that
 * runs out sets CSA2_DEVERR_TIMEOUT in the call's error word, the kernel frees
 * its tensor memory and returns, and the context stays usable.  This launches
 * one warp that holds 32 TMEM columns across the same bounded wait on an
 * mbarrier that one arrival completes (complete = 1: the wait succeeds, no bit
 * is set) or that nothing completes (complete = 0: the wait gives up after
 * `iters` polls of at most ~1 ms each and sets the TIMEOUT bit), so that a host
 * can see the bit arrive and keep using the device.  iters 1..64; err_word:
 * device int32, 4-byte aligned, required (OR-ed into, never cleared).
 * Asynchronous on `stream` like every other call.
 */
csa2_status csa2_bounded_wait_check(int32_t iters, int32_t complete, int32_t *err_word, csa2_stream_t stream);

/*
 * csa2_set_phase_events: measurement helper.  events: n_events cudaEvent_t
 * (created by the caller, owned by it) that this thread's next
 * csa2_prefill_chunk calls record on their stream, in order, at the phase
 * boundaries: the start, append + window rows done, then per block of queries
 * scored, selected, attended (each call restarts at the first event; events
 * beyond n_events are not recorded).  NULL / 0 stops the recording.
 * csa2_phase_events_recorded() gives how many the last call recorded.
 */
csa2_status csa2_set_phase_events(void *const *events, int32_t n_events);
int32_t csa2_phase_events_recorded(void);

/* Status text, and the thread-local detail of this thread's last failure. */
const char *csa2_status_string(csa2_status status);
const char *csa2_last_error_detail(void);
/* Library version, major*10000 + minor*100 + patch. */
int32_t csa2_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_H */
