/*
 * ai_index.h - C ABI of the causal IVF top-k key selection library
 * (libai_index.so, sm_100a).
 *
 * What it computes.  For every query of a chunked causal prefill, the top-k
 * keys under the DSA indexer score
 *     I(q, s) = sum_h w_h * ReLU(q_h . k_s),
 * selected through a causal inverted-file index over the indexer keys, as
 * described on the pages titled "AttentionIndex: Accelerating Learned Sparse
 * Attention with a Causal Inverted-File Index" (paper-daily.com explainer;
 * kurate.org review).  Sections cited below are those of the explainer.
 *
 * Conventions for every call.
 *  - Pointers named *_dev are CUDA device pointers owned by the caller; the
 *    library never frees them.  Pointers named *_host are host memory.
 *  - All work is enqueued on the handle's main stream (given at create time)
 *    and is asynchronous unless stated otherwise; call ai_sync() to wait
 *    and to collect device-side error flags.
 *  - Return value: AI_OK (0) or a negative AI_ERR_* code; ai_last_error()
 *    gives a message for the calling thread.  A call that fails leaves the
 *    index unchanged unless stated otherwise.
 *  - Layouts are row-major and dense: keys [n, d], queries [T, H, d],
 *    head weights [T, H] float32, outputs [T, k] int32.  With bf16 queries
 *    the query and head-weight pointers must be 16-byte aligned (they are
 *    read by bulk tensor copies); AI_ERR_ARG otherwise.
 *  - One handle is one (request, layer) index; handles are independent and
 *    must not be used from two threads at once.
 */
#ifndef AI_INDEX_H_
#define AI_INDEX_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ errors */
#define AI_OK 0
#define AI_ERR_ARG (-1)          /* invalid argument, shape or dtype            */
#define AI_ERR_OOM (-2)          /* device allocation failed, or max_keys hit  */
#define AI_ERR_CAUSALITY (-3)    /* a query position beyond the appended keys  */
#define AI_ERR_DEVICE_CHECK (-4) /* a kernel flagged an out-of-range id/offset */
#define AI_ERR_TIMEOUT (-5)      /* a bounded device wait or host wait ran out */
#define AI_ERR_CUDA (-6)         /* a CUDA runtime call failed                 */
#define AI_ERR_STATE (-7)        /* call not valid in the current state        */

/* ------------------------------------------------------------ dtypes */
#define AI_FP32 0     /* float32                                              */
#define AI_BF16 1     /* bfloat16 bits (uint16)                               */
#define AI_FP8E4M3 2  /* OCP FP8 E4M3 codes (uint8) + one float32 scale per key */

typedef struct ai_index* ai_handle;

/* Index configuration.  Field names follow the pages' notation.           */
typedef struct ai_config {
  int32_t d;                   /* key / query head dimension                 */
  int32_t H;                   /* indexer heads                              */
  int32_t key_dtype;           /* AI_FP32 | AI_BF16 | AI_FP8E4M3             */
  int32_t q_dtype;             /* AI_FP32 (only with AI_FP32 keys) | AI_BF16 */
  int32_t n_sinks;             /* S: first keys, always candidates, never clustered */
  int32_t window;              /* W: open keys sealed together               */
  int32_t clusters_per_window; /* m                                          */
  int32_t cluster_cap;         /* size cap at seal; 0 -> ceil(W / m)         */
  int32_t refit_period;        /* R (multiple of W); 0 = never refit         */
  int32_t refit_new_seeds;     /* seeds per refit; 0 -> R * m / W            */
  int32_t refit_seed_window;   /* seeds come from the last keys; 0 -> R      */
  int32_t seal_iters;          /* k-means passes at seal; 0 -> 10            */
  int32_t async_refit;         /* 1: refit runs on an internal side stream   */
  int32_t max_query_chunk;     /* largest T passed to route/exhaustive calls */
  int32_t max_budget;          /* largest C passed to ai_route_refine        */
  int32_t max_k;               /* largest k: <= 2048 (bf16 / fp8 keys),      */
                               /* <= 4096 (fp32 keys)                        */
  int64_t max_keys;            /* capacity of the key store                  */
  uint64_t seed;               /* seed of the refit seed draws (SplitMix64)  */
  const float* encoder_weights_host; /* NULL: plain mean representatives.   */
  /* Else the correction encoder's float32 weights, packed in this order:
   * A [d,d], a [d], B1 [d, 3d+1], b1 [d], B2 [d,d], b2 [d] (copied at create). */
  int32_t block_routing;       /* 0: the inverted-file index (k-means seal,  */
  /* refit).  1: the contiguous-block baseline the explainer compares against
   * ("它到底在解决什么问题？", HiSA): a sealed window is cut into m blocks of
   * consecutive keys, block j = keys [lo + floor(jW/m), lo + floor((j+1)W/m)),
   * each represented by its member mean; no refit (refit_period must be 0),
   * no encoder.  Routing, candidate fill, rescore and top-k are unchanged.  */
} ai_config;

/* Create an index.  `cuda_stream` is the main stream (cudaStream_t, may be
 * NULL for the legacy default stream).  Allocates the key store and all
 * device scratch sized from the config.  Errors: AI_ERR_ARG, AI_ERR_OOM,
 * AI_ERR_CUDA.  On success *out is a new handle.                           */
int ai_index_create(const ai_config* cfg, void* cuda_stream, ai_handle* out);

/* Free a handle and everything it owns (waits for its streams first).     */
int ai_index_destroy(ai_handle h);

/* Insert (explainer, "索引怎么边算边建？" item 1).  Appends n keys to the
 * append-only store; they are candidates of every later query at once (the
 * open window).  keys_dev: [n, d] in the key dtype (fp8: codes);
 * scales_dev: [n] float32 per-key scales for AI_FP8E4M3, else NULL.
 * Also publishes a pending refit first (see ai_refit).  Errors: AI_ERR_ARG,
 * AI_ERR_OOM (store full).                                                */
int ai_append_keys(ai_handle h, const void* keys_dev, const float* scales_dev, int64_t n);

/* Seal (explainer, "索引怎么边算边建？" item 2).  Clusters every complete
 * W-window of open keys into m size-capped k-means clusters and appends
 * them; each seal creates a version whose open window starts after the
 * sealed keys.  Whenever the number of sealed keys reaches a multiple of R
 * a refit is started (see ai_refit).  *version_out (nullable) receives the
 * newest version number.                                                  */
int ai_seal(ai_handle h, int64_t* version_out);

/* Refit (explainer, "索引怎么边算边建？" item 3).  One warm-started assign +
 * update pass over all sealed keys [S, n_r): previous refit centres plus
 * new seeds drawn from the last keys, Hamerly bounds, member means.  Runs
 * on the side stream when async_refit = 1.  The result becomes the index
 * base at the next ai_append_keys or ai_publish call (a version with
 * watermark n_r).  n_new_seeds / seed_window: 0 -> config values.         */
int ai_refit(ai_handle h, int32_t n_new_seeds, int32_t seed_window, int64_t* version_out);

/* Make a pending refit the index base now (waits on the side stream from
 * the main stream, not from the host).  No-op without a pending refit.     */
int ai_publish(ai_handle h);

/* Route + refine (explainer, "查询时怎么挑候选？").  For the T queries at
 * positions pos0 .. pos0+T-1: each query t uses the newest version whose
 * keys all lie in its prefix, scores every visible cluster representative,
 * fills C candidate slots with the sinks, the open window [n_v, t] and
 * whole member lists in rank order (score desc, cluster id asc; the last
 * list is truncated), rescores the candidates exactly and writes the top k
 * ids to out_dev[T, k] sorted by score descending, ties by key id
 * ascending, then -1 padding (fewer than k candidates).  q_dev: [T, H, d]
 * in q_dtype; w_dev: [T, H] float32; out_scores_dev: [T, k] float32 (the
 * scores of those ids, -inf on padding) or NULL.
 * Limit: at most 2048 clusters of one query can reach its budget (the
 * clusters ranked in shared memory).  Clusters hold ~W/m keys after a seal,
 * so this binds only when C / (smallest cluster size) exceeds 2048; a
 * query over the limit ranks only 2048 of them and ai_sync then reports
 * AI_ERR_DEVICE_CHECK.
 * Errors: AI_ERR_ARG (T, k, C beyond the create-time maxima),
 * AI_ERR_CAUSALITY (pos0 + T - 1 >= appended keys).                        */
int ai_route_refine(ai_handle h, const void* q_dev, const float* w_dev, int64_t pos0,
                    int32_t T, int32_t k, int32_t C, int32_t* out_dev, float* out_scores_dev);

/* Sharded rescore for a cluster-sharded, several-GPU deployment (the
 * review's "tensor-parallel index ownership", Impact Assessment: Core
 * Contribution item 3; the explainer, 我认为它的局限 item 2, names the
 * cross-GPU synchronisation).  Every rank holds the same index (maintenance
 * is deterministic); for each query it builds the same candidate list and
 * rescores only its share: the contiguous range of the list's 128-slot
 * tiles with index shard of n_shards.  It writes that share's top k to
 * out_dev / out_scores_dev [T, k] (both required), in (score desc, id asc)
 * order, -1 / -inf padded.  The shards' lists hold disjoint ids and the
 * union of their top k holds the query's top k: gathering the n_shards
 * partial results and merging them with ai_merge_topk gives exactly
 * ai_route_refine's output.  bf16 / fp8 keys (pipelined refine kernels)
 * only; n_shards = 1 is ai_route_refine.  Errors as ai_route_refine, and
 * AI_ERR_ARG for a bad shard.                                              */
int ai_route_refine_shard(ai_handle h, const void* q_dev, const float* w_dev, int64_t pos0,
                          int32_t T, int32_t k, int32_t C, int32_t shard, int32_t n_shards,
                          int32_t* out_dev, float* out_scores_dev);

/* Merge n_parts partial top-k results per query: ids_dev / scores_dev are
 * [n_parts, T, k] (ids -1 where a part has fewer than k); writes the top k
 * of each query's union by (score desc, id asc) to out_dev [T, k] (and
 * out_scores_dev, nullable), -1 padded.  The parts must hold disjoint ids.
 * Enqueued on cuda_stream; needs no handle and allocates nothing.  Limits:
 * k <= 2048, n_parts * k <= 19,840 (AI_ERR_ARG).                          */
int ai_merge_topk(const int32_t* ids_dev, const float* scores_dev, int32_t n_parts, int32_t T,
                  int32_t k, int32_t* out_dev, float* out_scores_dev, void* cuda_stream);

/* Exhaustive selection (explainer, "它到底在解决什么问题？": the indexer
 * scores every key s <= t).  Same arguments and output order as
 * ai_route_refine (score descending, ties by id ascending, -1 padding).
 * The in-library baseline.                                                */
int ai_select_exhaustive(ai_handle h, const void* q_dev, const float* w_dev, int64_t pos0,
                         int32_t T, int32_t k, int32_t* out_dev, float* out_scores_dev);

/* Wait for all work of the handle (both streams) and report device-side
 * error flags: AI_ERR_DEVICE_CHECK or AI_ERR_TIMEOUT (flags are cleared).  */
int ai_sync(ai_handle h);

/* Message of the last error on this thread ("" if none).                  */
const char* ai_last_error(void);

/* -------------------------------------------------------- inspection */
typedef struct ai_stats {
  int64_t n_keys;        /* appended keys                                   */
  int64_t n_sealed;      /* sealed windows                                  */
  int64_t n_clusters;    /* clusters in the published array                 */
  int64_t n_versions;    /* versions in the published table                 */
  int64_t n_refits;      /* refits started                                  */
  int64_t refit_pending; /* 1 if a refit awaits publication                 */
  int64_t base_watermark;/* n_r of the published base (0 = none)            */
  int64_t last_refit_scanned; /* keys fully scanned by the last finished refit */
  int64_t last_refit_rechecked; /* of those, keys re-decided in float64 (near ties) */
} ai_stats;
int ai_get_stats(ai_handle h, ai_stats* out);

/* Copy the published index to host memory (synchronous).  Any pointer may
 * be NULL.  offsets_host [n_clusters + 1] (member offsets, relative),
 * members_host [offsets[n_clusters]], reps_bf16_host [n_clusters, d],
 * centroids_host [n_clusters, d] float64, version_nc_host / version_nv_host
 * [n_versions] (visible clusters, open-window start).                      */
int ai_export_index(ai_handle h, int32_t* offsets_host, int32_t* members_host,
                    uint16_t* reps_bf16_host, double* centroids_host, int64_t* version_nc_host,
                    int64_t* version_nv_host);

/* Debug: the candidate lists [T, C] (-1 padded) and cluster scores
 * [T, n_clusters] that ai_route_refine would use for these queries.        */
int ai_debug_candidates(ai_handle h, const void* q_dev, const float* w_dev, int64_t pos0,
                        int32_t T, int32_t C, int32_t* cand_dev, float* cluster_scores_dev);

/* Debug: the full indexer score matrix out_dev[T, n_keys] (float32, -inf
 * where key position > query position) computed by the exhaustive kernels. */
int ai_debug_scores(ai_handle h, const void* q_dev, const float* w_dev, int64_t pos0, int32_t T,
                    float* out_dev);

/* Checkpoint / rollback of the index state (host counters, version table,
 * active cluster buffer, per-key refit bounds and the last centre drifts).  Rollback forgets keys
 * appended after the checkpoint (they must be appended again).  Fails with
 * AI_ERR_STATE while a refit is pending at checkpoint time.               */
int ai_checkpoint(ai_handle h);
int ai_rollback(ai_handle h);

/* ----------------------------------------------------------- profiling */
/* Phase timing with CUDA events recorded on the stream each phase runs on
 * (refit: the side stream when async).  Off by default.                    */
#define AI_PHASE_ROUTE 0       /* cluster-score GEMM                          */
#define AI_PHASE_REFINE 1      /* candidate fill + rescore + top-k kernel     */
#define AI_PHASE_SEAL 2        /* seal k-means (+ encoder)                    */
#define AI_PHASE_REFIT 3       /* refit kernels (+ encoder)                   */
#define AI_PHASE_PUBLISH 4     /* wait for the refit + tail copy              */
#define AI_PHASE_EXH_SCORES 5  /* exhaustive score GEMM                       */
#define AI_PHASE_EXH_TOPK 6    /* exhaustive row top-k                        */
#define AI_PHASE_ORDER 7       /* route+refine output ordering (tensor core)  */
#define AI_N_PHASES 8
int ai_profile_enable(ai_handle h, int enable);
/* Waits for the handle's streams, then writes the summed milliseconds and
 * the number of timed launches per phase (arrays of AI_N_PHASES, nullable)
 * since the last read, and resets them.                                   */
int ai_profile_read(ai_handle h, double* ms_out, int64_t* launches_out);
/* Number of kernels this library has launched in the process.             */
long long ai_kernel_launches(void);

/* fp8 store helper: per-key scale = amax / 448 and E4M3 codes (round to
 * nearest even, saturating) from bf16 keys [n, d].  Enqueued on
 * cuda_stream.                                                            */
int ai_quantize_fp8(const uint16_t* keys_bf16_dev, int64_t n, int32_t d, uint8_t* codes_dev,
                    float* scales_dev, void* cuda_stream);

/* ----------------------------------------------- allocation-free variant */
/* Exhaustive selection for callers that cannot allocate device memory (for
 * example a server whose memory all comes from its own pre-reserved pool, or
 * a latency-critical path that must not hit the implicit synchronisation of
 * cudaMalloc / cudaFree).  No counterpart in the paper: it is a deployment
 * convenience with the same results as ai_select_exhaustive on the same
 * keys.  It needs no handle and calls no allocator: its only scratch is a
 * fixed 16 MiB device array inside the library, present on every device
 * that loads the library until the process exits.
 *   keys_dev: [n_keys, d] keys owned by the caller: AI_BF16 (d = 128,
 *     H in {32, 64}, bf16 queries) or AI_FP32 (fp32 queries); n_keys at
 *     most 1,048,576 (AI_ERR_ARG beyond); k at most 4096.
 *   q_dev [T, H, d], w_dev [T, H], pos0, T, k, out_dev [T, k],
 *   out_scores_dev [T, k] or NULL: as for ai_select_exhaustive (same
 *     output order).
 *   status_dev: NULL, or a device int32 that receives, in stream order
 *     after the call's kernels, the device flags they raised: 0 when clean,
 *     else an OR of AI_DEVFLAG_* (the handle-based calls report the same
 *     flags through ai_sync).  A nonzero status means the output is not
 *     valid.
 * Enqueued on cuda_stream.  The first call on a device looks up the
 * array's device address (make it before any stream capture).  All calls
 * share the array: calls whose work overlaps on the GPU (other streams,
 * other threads) race and must be serialised by the caller.              */
#define AI_DEVFLAG_TIMEOUT 1   /* a bounded wait inside a kernel ran out     */
#define AI_DEVFLAG_RANGE 2     /* an id or offset was out of range           */
#define AI_DEVFLAG_CAPACITY 4  /* a per-CTA buffer would have overflowed     */
int ai_select_exhaustive_noalloc(const void* keys_dev, int32_t key_dtype, int64_t n_keys,
                                 int32_t d, int32_t H, const void* q_dev, const float* w_dev,
                                 int64_t pos0, int32_t T, int32_t k, int32_t* out_dev,
                                 float* out_scores_dev, int32_t* status_dev, void* cuda_stream);

/* ------------------------------------------------ refine kernel variant */
/* Selects the kernel that runs route+refine on the tensor-core path (bf16
 * or fp8 keys) for later ai_route_refine / ai_debug_candidates calls on h.
 * All variants compute the same result; this exists so tests can cover
 * each one.  kernel: 0 = chosen by occupancy (the default), 1 = one query
 * at a time per CTA with the candidate list in shared memory, 2 = the same
 * with the list in global scratch, 3 = pipelined (the candidate build and
 * the top-k of neighbouring queries overlap the rescore of the current
 * one), 4 = pipelined with one TMEM score buffer (the epilogue's first
 * score store waits for the previous query's top-k; the default for
 * budgets where two buffers would cost the second CTA per SM).  A variant
 * whose shared memory or TMEM need does not fit the configuration makes
 * those calls fail with AI_ERR_CUDA.  Returns AI_OK, or AI_ERR_ARG for a
 * null handle or a kernel outside 0..4.                                   */
int ai_debug_refine_kernel(ai_handle h, int32_t kernel);

/* Parts per query for later ai_route_refine calls on h (tensor-core path,
 * pipelined refine kernels).  A chunk of T queries with 2 * T at most the
 * pipelined kernel's CTA count (two per SM) would leave most SMs idle, one
 * CTA gathering each query's whole candidate list; instead each list's
 * 128-slot tiles are divided among `split` CTAs (contiguous ranges, at
 * least two tiles each) and their partial top-k merged by a second kernel
 * into the documented output order.  Every tile, and so every score, is
 * the same as undivided: results are identical either way.  split: 0 =
 * chosen by chunk size (the default: up to 8 parts, and at most the CTA
 * count divided by T), 1 = never divide, 2..8 = at most that many parts.
 * Returns AI_OK, or AI_ERR_ARG for a null handle or split outside 0..8.   */
int ai_debug_refine_split(ai_handle h, int32_t split);

/* The refine kernel ai_route_refine launches on h for budget C:
 * *kernel_out = 0 for the fp32 (SIMT) path, else the tensor-core variant
 * as numbered for ai_debug_refine_kernel (1 to 4; the forced one if
 * set).  Host-only: launches nothing.  AI_ERR_ARG for a null argument or
 * C outside 1 .. max_budget.                                              */
int ai_refine_kernel_choice(ai_handle h, int32_t C, int32_t* kernel_out);

/* -------------------------------------------- attention over the keys */
/* What a layer does with the selection: its queries attend over the keys and
 * values of the request, which live in a paged cache next to the index.  No
 * counterpart on the pages, which end at the indices; the formulas are
 * ordinary softmax attention:
 *     o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  s_j = scale * (q . k_j),
 *     lse = m + ln sum_j e^(s_j - m),                 m = max_j s_j,
 * over the keys j that the row sees.  A row that sees no key, or whose scores
 * are all -inf, gives zeros and lse = -inf.  Keys and values that a row does
 * not see have no influence on it, whatever they hold (NaN included).
 * Forward only: the library selects and serves; it has no training path.
 * n_heads query heads share n_kv_heads key heads in groups of
 * n_heads / n_kv_heads consecutive heads.  Queries and outputs are bf16,
 * sums and statistics float32, weights rounded to bf16 for the product with
 * v (fp8 caches: to f16, 11 bits down to 2^-15 of a row's largest weight and
 * below that to within 2^-26 of it); head_dim is 64 or 128, scale finite and
 * not negative.
 * The calls are enqueued on cuda_stream, allocate nothing and may be captured;
 * they need no handle.  Calls whose work may overlap (two streams, two graphs)
 * need a workspace each.                                                  */

/* A paged cache, all of it device memory of the caller's:
 *   k, v        [n_layers, n_pages, page_size, n_kv_heads, head_dim] in
 *               dtype (AI_BF16, or AI_FP8E4M3 codes), 16-byte aligned
 *   k_scale,    [n_layers, n_pages, page_size, n_kv_heads] float32, one per
 *   v_scale     token and head (AI_FP8E4M3; v_scale not negative), else NULL
 *   tables      [n_seqs, max_pages] int32: page p of a sequence holds its
 *               tokens [p * page_size, (p + 1) * page_size)
 *   lens        [n_seqs] int32: tokens of each sequence
 *   refs        [n_pages] int32: sequences that hold the page, 0 = free (only
 *               the ai_cache_* calls use it; may be NULL for ai_attend_* and
 *               ai_cache_write)
 *   status      an int32 that collects AI_DEVFLAG_* bits, or NULL: the
 *               device's own word, which ai_status_read reads.  RANGE for an
 *               id, sequence or page out of range (skipped, no access),
 *               CAPACITY where pages ran out (that sequence is unchanged),
 *               TIMEOUT where a wait inside a kernel ran out (the call's
 *               output is not valid)
 * n_pages at most 2^20; n_pages * page_size and max_pages * page_size below
 * 2^31.                                                                   */
typedef struct ai_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int32_t* status;
  int32_t dtype, n_layers, n_pages, page_size, n_kv_heads, head_dim;
  int32_t n_seqs, max_pages;
} ai_cache;

/* Causal attention over packed prompts.  Sequence b's queries are rows
 * [cu_q[b], cu_q[b+1]) of q, its keys rows [cu_k[b], cu_k[b+1]) of k and v
 * (device int32 [n_seqs + 1], ascending, within [0, total]).  The last query
 * sees the last key: query i of Lq sees keys j <= Lk - Lq + i (so a chunk
 * whose prefix precedes it in k and v is attended as it stands; with
 * Lk < Lq the first rows see nothing).  q [total_q, n_heads, head_dim] and
 * k, v [total_k, n_kv_heads, head_dim] bf16, the last dimension dense; the
 * strides (in elements) of the first two are given as {token, head} pairs
 * and are positive multiples of 8, bases 16-byte aligned.  out [total_q, n_heads,
 * head_dim] bf16 and lse [total_q, n_heads] float32 (nullable) are dense;
 * rows that belong to no sequence stay as they were.  status_dev: an int32
 * that collects AI_DEVFLAG_* bits, or NULL as in ai_cache (RANGE: cu_q / cu_k not as above,
 * nothing out of range is touched but the output is not valid; TIMEOUT as
 * for ai_cache).
 * Limits: n_heads / n_kv_heads at most 128; total_q and total_k at most
 * 2^31 - 257.                                                             */
int ai_attend_prompt(const void* q_dev, const int64_t* q_strides, const void* k_dev,
                     const int64_t* k_strides, const void* v_dev, const int64_t* v_strides,
                     const int32_t* cu_q_dev, const int32_t* cu_k_dev, int32_t n_seqs,
                     int32_t total_q, int32_t total_k, int32_t n_heads, int32_t n_kv_heads,
                     int32_t head_dim, float scale, void* out_dev, float* lse_dev,
                     int32_t* status_dev, void* workspace_dev, int64_t workspace_bytes,
                     void* cuda_stream);

/* Bytes of workspace that ai_attend_prompt needs for these sizes, on the
 * current device: 0 unless there are too few queries to fill it and the
 * sequences average 1024 keys or more; then the keys are divided.         */
int ai_attend_prompt_workspace(int32_t n_seqs, int32_t total_q, int32_t total_k, int32_t n_heads,
                               int32_t n_kv_heads, int32_t head_dim, int64_t* bytes_out);

/* Bytes of workspace that ai_attend_cached and ai_attend_selected need for
 * these heads (whatever the lengths).                                     */
int ai_attend_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int64_t* bytes_out);

/* One new token per sequence (decode): row r of q [n_rows, n_heads,
 * head_dim] attends over all lens tokens of sequence seqs[r] of the cache.
 * seqs_dev NULL: row r is sequence r (n_rows = n_seqs).                   */
int ai_attend_cached(const ai_cache* cache, int32_t layer, const void* q_dev, int32_t n_rows,
                     int32_t n_heads, const int32_t* seqs_dev, float scale, void* out_dev,
                     float* lse_dev, void* workspace_dev, int64_t workspace_bytes,
                     void* cuda_stream);

/* Attention over selected keys: row t of q [T, n_heads, head_dim] attends
 * over the tokens ids_dev[t, 0..k) (what ai_route_refine writes) of sequence
 * seqs[t]; negative ids are no keys, an id that occurs twice counts twice.
 * seqs_dev NULL: every row is the cache's only sequence (n_seqs = 1), or row
 * t is sequence t (n_seqs = T).                                           */
int ai_attend_selected(const ai_cache* cache, int32_t layer, const void* q_dev,
                       const int32_t* ids_dev, int32_t T, int32_t k, int32_t n_heads,
                       const int32_t* seqs_dev, float scale, void* out_dev, float* lse_dev,
                       void* workspace_dev, int64_t workspace_bytes, void* cuda_stream);

/* ------------------------------------------------- pages of the cache */
/* All state is device memory and every change is made in stream order, so
 * these calls may be captured too.  New pages are the lowest free ones, in
 * the order of the list.  A sequence with lens = 0 is empty.  What a call
 * refuses (bad index, a sequence listed twice, pages exhausted) is flagged in
 * cache->status and left unchanged; the rest of the list is done.  (Released
 * twice is not refused: the second time the sequence is empty.)           */

/* Bytes of workspace for a call with an n-entry list (ai_cache_compact: 0). */
int ai_cache_workspace(const ai_cache* cache, int32_t n, int64_t* bytes_out);

/* Lengthen sequence seqs[i] by counts[i] tokens, taking pages as needed.  A
 * sequence is lengthened if it needs no page, or if the pages it and the
 * listed ones before it need are there.  The new tokens' contents come with
 * ai_cache_write, once per layer.                                         */
int ai_cache_extend(const ai_cache* cache, const int32_t* seqs_dev, const int32_t* counts_dev,
                    int32_t n, void* workspace_dev, int64_t workspace_bytes, void* cuda_stream);

/* Write the keys and values [n_tokens, n_kv_heads, head_dim] bf16 (dense) of
 * one layer: rows [cu[i], cu[i+1]) become the last cu[i+1] - cu[i] tokens of
 * sequence seqs[i] (fp8: quantised as by ai_quantize_fp8, per token and
 * head).  cu_dev int32 [n + 1], ascending; rows outside are not read.  Rows
 * before a sequence's first token (cu asks for more than it has) are left out
 * and flagged (RANGE).  Where cache->refs is given, a sequence whose rows
 * reach a page that another one holds too is refused as a whole (RANGE);
 * without it such a write changes them all.
 * Write a sequence's tokens in every layer before it is forked.           */
int ai_cache_write(const ai_cache* cache, int32_t layer, const void* k_dev, const void* v_dev,
                   const int32_t* seqs_dev, const int32_t* cu_dev, int32_t n, int32_t n_tokens,
                   void* cuda_stream);

/* Make the empty sequence dst[i] a copy of sequence src[i]: full pages are
 * shared, the filled slots of a part page are copied to a fresh page.  All
 * forks of a call see the state before it.                                */
int ai_cache_fork(const ai_cache* cache, const int32_t* src_dev, const int32_t* dst_dev, int32_t n,
                  void* workspace_dev, int64_t workspace_bytes, void* cuda_stream);

/* Release sequences: their pages lose one reference each, their table rows
 * become -1, their lengths 0.                                             */
int ai_cache_free(const ai_cache* cache, const int32_t* seqs_dev, int32_t n, void* cuda_stream);

/* Move the live pages to the front of the cache: with L live pages, the i-th
 * live page at or behind L moves to the i-th free page before L (all layers);
 * tables and refs follow.                                                 */
int ai_cache_compact(const ai_cache* cache, void* workspace_dev, int64_t workspace_bytes,
                     void* cuda_stream);

/* The AI_DEVFLAG_* bits that attention and cache calls without a status word
 * have raised on the current device since the last read (of the calls whose
 * work cuda_stream is behind: it waits for that stream), and clears them.
 * Not to be called while a stream is captured.  AI_ERR_ARG for a null
 * output, AI_ERR_CUDA on a CUDA error.                                    */
int ai_status_read(int32_t* bits_out, void* cuda_stream);

/* ------------------------------------------------- failure-path test hook */
/* Runs the library's bounded wait against a barrier that nothing completes
 * (the pages have no counterpart: this exists to test failure detection).
 * One thread polls an mbarrier phase at most spin_limit times (1 .. 2^26),
 * then records the timeout in a device status word and returns, exactly as
 * a kernel whose producer never arrives would.  Enqueued on cuda_stream and
 * waited for.  *status_out receives the device status flags (bit 0 =
 * timeout).  Returns AI_OK when the wait ran out and was reported,
 * AI_ERR_ARG for a bad limit or null output, AI_ERR_CUDA on a CUDA error.  */
int ai_debug_wait_timeout(int32_t spin_limit, int32_t* status_out, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* AI_INDEX_H_ */
