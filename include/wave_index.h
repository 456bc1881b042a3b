/*
 * wave_index.h -- C ABI of the GB300 wave-index hot path.
 *
 * RetroInfer treats the KV cache as a vector store that each decode step
 * queries (RetroInfer abstract; summaries de/fr/zh section 2.A).  This library
 * builds that store's index at prefill -- segmented spherical k-means over
 * the keys of every (sequence, layer, kv head), with per-cluster counts, mean
 * keys and value sums -- and runs the decode-time tripartite attention:
 * steady zone (sinks + local window) and the top-k retrieved clusters exactly,
 * every other cluster estimated from its mean key, count and value sum, the
 * zones merged by log-sum-exp.
 *
 * Conventions for every entry point:
 *   - All tensors are row-major and contiguous.  bf16 tensors are passed as
 *     raw 16-bit patterns (uint16_t / void*).
 *   - "device" pointers must be CUDA device memory of the current device
 *     (cudaMalloc / torch); "host" pointers plain host memory; "any" pointers
 *     either (copied with cudaMemcpyDefault, so they must be UVA-addressable).
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Work is
 *     enqueued on it; outputs are valid once the stream has been synchronised,
 *     unless stated otherwise.
 *   - Every call returns WI_OK (0) or a negative WI_E* code and then leaves a
 *     thread-local message readable with wi_last_error().  No call aborts,
 *     exits, throws across the ABI or traps on the device.  On error an
 *     output handle is set to NULL.
 *   - Head size d must be 128.  Query head h attends with kv head h / g,
 *     g = n_q_heads / n_kv_heads.  A "unit" is one (sequence b, layer l,
 *     kv head h), numbered u = (b * layers + l) * n_kv_heads + h.
 */
#ifndef WAVE_INDEX_H
#define WAVE_INDEX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  WI_OK = 0,
  WI_EINVAL = -1,       /* bad argument: shape, null pointer, d != 128, k > C, ... */
  WI_ENOMEM = -2,       /* a device or host allocation failed */
  WI_ECUDA = -3,        /* a CUDA runtime call failed (message names it) */
  WI_EUNSUPPORTED = -4, /* valid but not supported by this build */
  WI_EDEVICE = -5,      /* a kernel reported a violated invariant */
  WI_EFULL = -6         /* the append buffer is full */
};

typedef struct wi_index wi_index; /* opaque, library-owned */

/*
 * Shapes and method parameters.  Zones (summaries de/fr/zh 2.A): the steady
 * zone is positions [0, n_sink) and [n_ctx - local_window, n_ctx) plus every
 * token appended during decode; all other positions are clustered.
 * Segmented clustering (same sections): each run of seg_len positions is
 * clustered on its own into clusters_per_seg clusters (global id =
 * segment * clusters_per_seg + local id) by `iters` rounds of spherical
 * k-means (summary fr 2.A.2).  Retrieval budget (summary zh section 3):
 * k = budget_k if > 0, else ceil(budget_frac * C), C = all clusters of a unit;
 * capped at the unit's non-empty clusters at decode time.
 * Decode-time growth (an extension: the pages describe the index at prefill):
 * the index holds room for C = (n_ctx / seg_len + max_append / seg_len) *
 * clusters_per_seg clusters per unit; those of segments not grown yet are
 * empty, and the budget k counts only the clusters held so far.
 * Limits of this build (WI_EUNSUPPORTED beyond them): n_q_heads / n_kv_heads
 * <= 8, k <= 4096, seg_len <= 16384, C <= 65536 (room for growth included).
 */
typedef struct {
  int batch, layers, n_q_heads, n_kv_heads, head_dim; /* head_dim == 128 */
  long long n_ctx;        /* tokens per unit at build; a multiple of seg_len */
  int seg_len;            /* a multiple of 128, >= 128 */
  int clusters_per_seg;   /* multiple of 16 in [16, 512] dividing seg_len */
  int iters;              /* k-means rounds (assignments), >= 1 */
  int n_sink, local_window;
  int max_append;         /* capacity of the decode-time append buffer, >= 0; with max_append >=
                             seg_len the index also grows during decode (wi_decode_step) */
  double budget_frac;
  int budget_k;
  int valsum_bf16;        /* 0: decode reads the fp32 value sums; 1: it reads a bf16 copy made at
                             build / import (round to nearest even; half the estimation bytes) */
  int group_topk;         /* 0: each query head takes its own top-k; 1: the query heads of a kv head
                             share the top-k of their summed scores (each head keeps its own logits,
                             estimate and retrieved-term weights) */
  int reserved[1];        /* must be zero */
} wi_config;

/*
 * Build the index (prefill): segmented spherical k-means and the per-cluster
 * count, mean key and value sum of every unit (summaries de/fr/zh 2.A
 * "segmented clustering", fr 2.A.2 "spherical k-means", zh 2.A "precomputed
 * value sum").  k, v: device bf16 [batch][layers][n_kv_heads]
 * [n_ctx][128], caller-owned.  The library permutes their clustered rows IN
 * PLACE into cluster-contiguous order (cluster by cluster, by position inside
 * a cluster; steady rows stay where they are) and keeps pointing at them: the
 * caller keeps both alive and unmodified until wi_free.
 * init_centroids: NULL for the default seeding (the normalised key at the
 * start of each stride-(seg_len/clusters_per_seg) block of a segment), or
 * device bf16 [units][n_ctx/seg_len][clusters_per_seg][128] used as the
 * centroids of the first round (rows should be unit-norm).
 * Enqueues the build on `stream` and returns; *out is usable on that stream.
 */
int wi_build_index(const wi_config* cfg, void* k, void* v, const void* init_centroids, void* stream,
                   wi_index** out);

/*
 * Adopt an index computed elsewhere instead of clustering (e.g. by a CPU
 * reference).  counts: [units][Cb] int32, Cb = (n_ctx / seg_len) *
 * clusters_per_seg (the build's clusters); perm: [units][n_ctx - n_sink -
 * local_window] int32, the original position of every clustered slot in
 * cluster-contiguous order (slots of cluster j follow those of cluster j-1;
 * slot numbering starts at row n_sink); mu: bf16 [units][Cb][128] mean keys;
 * valsum: fp32 [units][Cb][128] value sums.  All four are "any" pointers and
 * are copied.  k, v as in wi_build_index (permuted in place by perm).
 * Returns WI_EINVAL if perm is not a bijection on the clustered positions
 * consistent with counts and segments (checked on the host).
 */
int wi_index_import(const wi_config* cfg, void* k, void* v, const int32_t* counts, const int32_t* perm,
                    const uint16_t* mu, const float* valsum, void* stream, wi_index** out);

/*
 * Copy the index out ("any" pointers; any of them may be NULL to skip it),
 * C = the clusters per unit from wi_index_shape (room for growth included).
 * counts [units][C], offsets [units][C+1] (row of the first slot of each
 * cluster; offsets[Cb] = n_ctx - local_window; a grown segment g's slots are
 * rows n_ctx + g*seg_len + slot), perm [units][n_ctx - n_sink - local_window
 * + (max_append / seg_len) * seg_len] (as in wi_index_import, then every grown
 * segment's seg_len slots; -1 where nothing has grown yet), mu bf16
 * [units][C][128], valsum fp32 [units][C][128].  Clusters not grown yet have
 * count 0 and zero mean key and value sum.  Asynchronous.
 */
int wi_index_export(const wi_index* ix, int32_t* counts, int32_t* offsets, int32_t* perm, uint16_t* mu,
                    float* valsum, void* stream);

/*
 * One decode step of the tripartite attention approximation (summaries
 * de/fr/zh 2.A: steady and retrieval zones exact, estimation zone from each
 * cluster's mean key, count and value sum, merged by log-sum-exp; zh section 3
 * for the ~1.8% retrieval budget).  q: device bf16 [batch][layers][n_q_heads][128], the
 * queries of the step (already rotated), 16-byte aligned; out: device fp32 [batch][layers]
 * [n_q_heads][128], attention output per query head.  Attention runs over
 * the current context: the n_ctx built tokens plus every token appended so
 * far.  If k_new and v_new (device bf16 [batch][layers][n_kv_heads][128]) are
 * non-NULL, that token is appended AFTER this step's attention; returns
 * WI_EFULL (nothing enqueued) when max_append tokens are already appended.
 * Appended tokens join the local window.  When an append leaves the window
 * holding local_window + seg_len rows (every seg_len appended tokens), the
 * step also grows the index: the window's oldest seg_len rows become one more
 * segment, clustered like a build segment (same seeds rule, iters rounds,
 * counts / mean keys / value sums; its rows copied, cluster-contiguous, into
 * library memory), its clusters take the next free ids and the budget is
 * recomputed for the clusters held.
 * Uses only library-owned scratch: no allocation and no host synchronisation.
 * Steps without append replay correctly from a captured CUDA graph (a graph
 * captured before a growth keeps attending over the grown index correctly:
 * the growth state lives in device memory).
 */
int wi_decode_step(wi_index* ix, const void* q, const void* k_new, const void* v_new, float* out, void* stream);

/*
 * wi_decode_step with HOST q / k_new / v_new / out: copies the inputs to the
 * device, runs the step, copies the output back and synchronises `stream`
 * before returning (out is valid on return).  Pinned host memory makes the
 * copies asynchronous DMA; pageable memory works but is slower.  A step with
 * pinned (device-mapped, 16-byte aligned) q and out, no append and decode
 * profiling off runs as one CUDA graph that the index captures for that pair
 * of buffers: a copy kernel reads q from host memory, the decode kernels run
 * and the final merge writes out straight to host memory.  The index owns a
 * stream and the graph until wi_free; a call with other buffers captures
 * again, and after a few such changes the index launches directly, as it
 * does for every other step.  Results are identical either way.
 */
int wi_decode_step_host(wi_index* ix, const void* q_host, const void* k_new_host, const void* v_new_host,
                        float* out_host, void* stream);

/*
 * Clusters retrieved by the last decode step: ids [units][g][k_max] int32
 * ("any"), ascending within each head, padded with -1; counts [units][g]
 * int32 ("any", may be NULL).  k_max is reported by wi_index_shape.
 */
int wi_last_selection(const wi_index* ix, int32_t* ids, int32_t* counts, void* stream);

/*
 * Full attention over every token the index holds: the dense comparator that
 * the wave index approximates (RetroInfer summaries de/fr/zh section 2.A; the
 * speed-up over it in zh section 3).  For every unit and query head,
 * out = softmax(q K^T / sqrt(128)) V over the unit's n_ctx context rows and
 * the tokens appended so far, with no index involved (the context rows are
 * read in the index's cluster-contiguous order; attention does not depend on
 * the order).  q: device bf16 [batch][layers][n_q_heads][128]; out: device
 * fp32, same layout (both caller-owned, q 16-byte aligned).  Uses the index's
 * own scratch: calls on one index must be ordered (one stream).  Stream-
 * ordered, asynchronous, no allocation, graph-capturable.  Fp32 accumulation.
 */
int wi_dense_decode(wi_index* ix, const void* q, float* out, void* stream);

/*
 * One kernel of the decode step alone (benchmarking aid: the duration of one
 * kernel in isolation, without events between kernels).  kernel 0: centroid
 * scores; 1: top-k with the estimation over all clusters; 2: exact attention
 * with the final merge.  Each kernel reads what the previous one wrote in the
 * last decode step of this index, so it repeats that step's work for its
 * part; q and out as in wi_decode_step (kernel 2 rewrites out).  Returns
 * WI_EINVAL before the index's first wi_decode_step.  Stream-ordered, no
 * allocation, graph-capturable.
 */
int wi_decode_kernel(wi_index* ix, int kernel, const void* q, float* out, void* stream);

/* Sizes of an index: units, clusters per unit C (room for decode-time growth
 * included), k_max (the budget for C clusters, the largest it can grow to),
 * group g, tokens appended so far (host-side count).  Any output pointer may
 * be NULL. */
int wi_index_shape(const wi_index* ix, int* units, int* clusters, int* k_max, int* group, int* appended);

/*
 * Launch layout of this index's decode kernels, fixed when the index is made
 * from the device's SM count: scores CTAs per unit, estimation CTAs per unit,
 * and exact-attention splits per head over the selected rows (one more CTA
 * takes the steady rows).  The environment variables WI_D1_CTAS_PER_UNIT,
 * WI_ESTIMATE_CTAS_PER_UNIT and WI_D3_SPLITS (positive integers), and
 * WI_ESTIMATE_FIRST (0 or 1: the estimation CTAs before the top-k CTAs in
 * their shared launch; default: when they fit in one wave), WI_D3_STAGE_ROWS
 * (32 or 64: rows per shared-memory stage of the exact-attention CTAs;
 * default 32 when all of them are resident at once, else 64) and
 * WI_ESTIMATE_DEPTH (2 or 3: value-sum tiles in flight per estimation CTA;
 * default 2 when the top-k and estimation CTAs fit in one wave, else 3),
 * read when the index is made, override the defaults.  Results do not depend on the
 * layout beyond float rounding order.  Any output pointer may be NULL.
 */
int wi_decode_layout(const wi_index* ix, int* score_ctas, int* estimate_ctas, int* exact_splits);

/*
 * One spherical k-means round on every segment, for per-round checking:
 * assignment of each clustered token against `centroids` (device bf16
 * [units][n_segments][clusters_per_seg][128]) written to assign (device int32
 * [units][n_ctx], global cluster id, -1 for steady positions), then the
 * updated centroids bf16(normalise(sum of normalised member keys)), empty
 * clusters unchanged, to new_centroids (device, same shape; may alias
 * centroids).  k: device bf16 keys as in wi_build_index (not modified).
 * Allocates and frees its own scratch on `stream`.
 */
int wi_kmeans_step(const wi_config* cfg, const void* k, const void* centroids, int32_t* assign,
                   void* new_centroids, void* stream);

/*
 * The default first-round centroids of every segment, for per-step checking
 * of the k-means initialisation (segmented spherical k-means: summaries
 * de/fr/zh 2.A, fr 2.A.2; seeding is not stated there, and this build takes
 * the first key of each stride-(seg_len/clusters_per_seg) block of the
 * segment, steady positions included): centroids[u][s][j] =
 * bf16(K[u][s*seg_len + j*stride] / |K[u][s*seg_len + j*stride]|), the
 * centroids that wi_build_index uses when init_centroids is NULL.
 * k: device bf16 keys as in wi_build_index (not modified); centroids: device
 * bf16 [units][n_segments][clusters_per_seg][128].  Asynchronous on `stream`.
 */
int wi_init_centroids(const wi_config* cfg, const void* k, void* centroids, void* stream);

/*
 * Per-kernel timing of decode steps (benchmarking aid).  After
 * wi_profile_begin(ix, max_steps), every decode step on this index records
 * CUDA events around each of its WI_NUM_DECODE_KERNELS kernels (centroid
 * scores; top-k with the retrieved clusters' estimation terms, sharing one
 * launch with the estimation over all clusters; exact attention with the
 * final merge) into slot
 * (step number % max_steps); steps captured into a CUDA graph record them on
 * every replay.  wi_profile_read synchronises the device and returns, per
 * kernel, the summed duration in milliseconds over the filled slots
 * (kernel_ms[WI_NUM_DECODE_KERNELS], may be NULL), the number of filled
 * slots, and the exact-zone rows processed by all decode steps since the
 * index was created, counted per query head (the bytes the exact-attention
 * kernel loads are rows * 512).
 * wi_profile_begin with max_steps = 0 turns recording off.
 */
#define WI_NUM_DECODE_KERNELS 3
int wi_profile_begin(wi_index* ix, int max_steps);
int wi_profile_read(wi_index* ix, double* kernel_ms, int* steps, unsigned long long* exact_rows);

/*
 * wi_kmeans_step without any device allocation (the paper has no
 * counterpart; this is an interface for callers that may not allocate).
 * A serving process usually gives nearly all GPU memory to its KV-cache
 * pool, and some hosts allow device memory only through their own arena;
 * such callers cannot let a clustering round call cudaMalloc.  Same
 * arguments, same results as wi_kmeans_step; its scratch is a fixed 8 MiB
 * device array that every GPU loading this library holds until the process
 * exits.  Problems that need more scratch (about 400K tokens in total at 512
 * clusters per 8192-token segment) return WI_EINVAL with a message.
 * All calls share the array: calls whose work overlaps on the GPU race on it
 * (order them on one stream).  Every call looks up the array's device
 * address with the caller's device current (no allocation), so a device
 * reset between calls is harmless.  Synchronises `stream` before returning.
 */
int wi_kmeans_step_noalloc(const wi_config* cfg, const void* k, const void* centroids, int32_t* assign,
                           void* new_centroids, void* stream);

/*
 * Timing of the build that made this index (CUDA events recorded on its
 * stream): whole build in ms, summed duration of its `iters` assignment
 * launches in ms, and their number.  Waits for the build to finish.  Returns
 * WI_EUNSUPPORTED for an index made by wi_index_import.  Any output may be NULL.
 */
int wi_index_build_stats(wi_index* ix, double* build_ms, double* assign_ms, int* assign_launches);

/* Synchronise the index's last stream and report a device-side invariant
 * violation recorded by any kernel since the last call (WI_EDEVICE). */
int wi_check_device(wi_index* ix);

/* Test hook: the failure path of the kernels' bounded waits, run on purpose.
 * Launches, on the current device, one kernel whose thread waits on a
 * shared-memory mbarrier that nothing ever completes, through the same
 * bounded wait the library's kernels use (it gives up after about 2^31 SM
 * cycles, ~1 s, records the timeout bit 16 in the kernel's error word and
 * returns), and synchronises the device.  On WI_OK, *device_error is the
 * kernel's error word (16 when the wait gave up) and *wait_returned 1 when the
 * wait returned without completion (2 if it had completed).  No fault, trap
 * or endless loop; the context stays usable.  Host outputs; errors:
 * WI_EINVAL (null pointer), WI_ENOMEM, WI_ECUDA. */
int wi_selftest_wait_timeout(int* device_error, int* wait_returned);

/*
 * Host memory tier: the wave buffer (summaries de/fr/zh section 2.B: a GPU
 * block cache of the KV blocks retrieval keeps returning to, LRU replacement
 * run by the CPU asynchronously, an execution buffer that feeds attention the
 * tokens from the steady zone, the cache and CPU memory).
 *
 * wi_tier_attach copies the index's permuted K and V (the caller's k / v,
 * device) to page-locked host memory owned by the library and the sink and
 * window rows to a device copy, and waits for `stream`; from then on no call
 * reads the caller's k / v, which the caller may free or reuse.  The host
 * rows are split into pages of 16 consecutive rows of a unit; each unit gets
 * `slots_per_unit` (0 .. pages per unit) page slots in device memory, empty at
 * first.  The exact-attention kernel of every later decode step copies each
 * retrieved row from its cached page or, if the page is not cached, straight
 * from host memory over the CPU-GPU link, and stamps the page with the step.
 * A replacement round takes the pages read since the previous round, in
 * increasing page order per unit: a cached page becomes the most recently
 * used; a page not cached is admitted (at most `admit_per_round` per unit and
 * round) into the lowest free slot, else into the slot of the least recently
 * used page unless that page was read in this same round, in which case the
 * round admits nothing more.  A round unmaps its victims on the decode stream,
 * fills their slots from host memory on a stream of its own and maps the new
 * pages on the decode stream once the fill has landed: decode never waits for
 * a round and never reads a slot being refilled.  With async != 0 a library
 * thread runs a round whenever it is idle after a decode step (on the newest
 * stamps); with async == 0 rounds run only in wi_tier_round.  Outputs do not
 * depend on where rows were read from: they equal the same index's outputs
 * without the tier bit for bit.
 * Needs an index that does not grow (max_append < seg_len) and fp32 value
 * sums (WI_EUNSUPPORTED otherwise).  Afterwards wi_dense_decode returns
 * WI_EUNSUPPORTED, and wi_decode_step refuses a stream being captured into a
 * graph.  Host memory: 2 * units * n_ctx * 256 bytes; device: 2 * units *
 * slots_per_unit * 4096 bytes plus 8 bytes per page for the tables.
 */
int wi_tier_attach(wi_index* ix, int slots_per_unit, int admit_per_round, int async, void* stream);

/* One replacement round now, on the calling thread, over the pages read by
 * every decode step enqueued so far; waits for a running round first and for
 * the round's own work before returning. */
int wi_tier_round(wi_index* ix, void* stream);

/* Counters of the tier since attach, after waiting for any running round and
 * the index's last stream: counters[6] = rounds, pages read (as the rounds saw
 * them), of which cached, of which not, pages admitted, pages evicted;
 * rows[2] = rows the exact-attention kernels copied from cached pages, from
 * host memory.  slots / pages: slots and pages per unit.  Outputs may be NULL. */
int wi_tier_stats(wi_index* ix, long long* counters, unsigned long long* rows, int* slots, int* pages);

/* Test hook: the tier's tables, host int32 [units][pages] each: the slot
 * holding each page (-1: not cached) and the last step that read it (-1:
 * none).  Waits like wi_tier_stats.  Either output may be NULL. */
int wi_tier_tables(wi_index* ix, int32_t* slot_of, int32_t* use);

/* The tier's replacement policy alone, on the host (no device involved), for
 * checking: a cache of `slots` pages out of `pages` for one unit.  wi_lru_round
 * runs one round for the pages in `touched` (any order, repeats ignored) at
 * round number t and writes the evictions and admissions, in the order it made
 * them, as (page, slot) pairs; each output array needs room for n entries (any
 * may be NULL).  wi_lru_new returns NULL for bad sizes. */
void* wi_lru_new(int pages, int slots, int admit_max);
int wi_lru_round(void* policy, const int32_t* touched, int n, long long t, int32_t* ev_pages, int32_t* ev_slots,
                 int* n_ev, int32_t* ad_pages, int32_t* ad_slots, int* n_ad);
void wi_lru_free(void* policy);

/*
 * Paged cache: where requests of different lengths are prefilled and decoded
 * before (or beside) an index.  One layer's keys and values live in two pools
 * of pages, k_pages and v_pages: device bf16 [n_pages][n_kv_heads][page_size]
 * [128], caller-owned, 16-byte aligned; a model's layers are pools of their
 * own that share one block table.  Row b of the block table (device int32
 * [max_batch or more][max_pages]) lists request b's pages: position p is row
 * p % page_size of page block_table[b][p / page_size], and its slot number is
 * page * page_size + p % page_size.  One page per request with page_size = n_ctx is
 * exactly the layout that wi_build_index takes.
 * A step: wi_paged_tables (lengths -> pages, slots, positions),
 * then in every layer wi_paged_write (norms and rotation, keys and values into
 * the pools) and wi_paged_attention; wi_paged_gather copies rows out into the
 * layout of wi_build_index or of wi_decode_step's k_new / v_new.
 *
 * Lengths and tables are read on the device only: no call synchronises, and
 * every call may be captured in a CUDA graph and replayed over new contents.
 * Kernels check what they read there (page numbers, lengths, offsets) before
 * they use it: a bad value is never followed, sets a bit that
 * wi_paged_check reports, and leaves the outputs of the request it belongs to
 * unspecified but inside their buffers.
 * Limits (WI_EUNSUPPORTED): 2^24 tokens in a step, 1024 query heads, and those
 * below.  No output shares memory with an input or another output (WI_EINVAL;
 * wi_paged_write has one exception).
 * A handle owns the attention's scratch and the error word and belongs to the
 * device that was current when it was made (WI_EINVAL on another): order the
 * attention calls on one handle (one stream; graphs that hold them one behind
 * the other, too); the other calls may overlap.
 */
typedef struct wi_paged wi_paged; /* opaque, library-owned */

typedef struct {
  int n_q_heads, n_kv_heads, head_dim; /* head_dim == 128; n_q_heads / n_kv_heads <= 8 */
  int page_size;          /* positions per page: a multiple of 16 */
  int n_pages;            /* pages in a pool; n_pages * n_kv_heads * page_size < 2^31 */
  int max_batch;          /* requests per call, at most; <= 4096 */
  int max_pages;          /* row width of the block table; max_pages * page_size < 2^31 */
  int rotary_dim;         /* elements of a head that are rotated: 0 (none) .. 128, a multiple of 8 */
  int interleaved;        /* 0: element i turns with i + rotary_dim / 2; 1: 2i with 2i + 1 */
  int reserved[3];        /* must be zero */
  double eps;             /* of the norms, > 0 */
  double rope_scale;      /* factor on both cosine and sine (1 for plain rotation) */
  const double* inv_freq; /* host, rotary_dim / 2 angles per position (radians), copied; NULL if none */
} wi_paged_config;

/* Make a handle on the current device (allocates the attention's scratch, about 270 KB per SM, and waits for the
 * default stream, on which it is cleared: the handle may be used on any stream at once). */
int wi_paged_create(const wi_paged_config* cfg, wi_paged** out);

/*
 * Positions of several axes (time, height and width of a picture's or a video's
 * tokens): pair i of the rotation turns by the position on axis[i].  axis: host
 * int32 [rotary_dim / 2], each in [0, n_axes), copied; n_axes in 1 .. 4, where 1
 * (as after wi_paged_create) takes axis away again.  From then on `positions` of
 * wi_paged_write and wi_paged_write8 is [n_axes][n_tokens].  A token whose first
 * axis' position is negative is padding; on other axes negative positions turn the
 * other way.  Calls that are in a graph keep the axes they were captured with.
 */
int wi_paged_axes(wi_paged* pc, int n_axes, const int32_t* axis);

/* Synchronise the device and report what kernels of this handle's calls found wrong
 * since the last check: WI_OK, or WI_EDEVICE with a message. */
int wi_paged_check(wi_paged* pc);

/* Release the handle.  NULL is a no-op.  Synchronises the device first. */
void wi_paged_free(wi_paged* pc);

/*
 * Pages, slots and positions of a step from its requests' lengths.  ctx_len,
 * new_len: device int32 [batch], positions in the cache before the step and
 * tokens that the step adds (0 allowed).  Request b holds the first
 * ceil(ctx_len / page_size) entries of its row; the pages that its new
 * positions need on top are taken from the end of free_pages (device int32,
 * the first *n_free of free_cap entries are free), request after request, a
 * request's own in increasing position, and entered in its row.  Other entries
 * of the block table stay as they were.  Written: kv_len [batch] = ctx_len +
 * new_len; q_start [batch + 1], the running sum of new_len (the step's tokens
 * lie request after request); slots and positions [n_tokens], of each token,
 * -1 for those behind the last; *n_free_out, the free pages that are left
 * (free_pages itself is not changed).  No output may share memory with an
 * input or another output (WI_EINVAL).
 * A length that is negative or beyond max_pages * page_size, more new tokens
 * than n_tokens, or more pages than *n_free: an error bit is set, and the step
 * takes no page and has no token (q_start all 0, kv_len = ctx_len, or 0 where
 * that is out of range).  Idempotent as long as *n_free and the lengths stay.
 */
int wi_paged_tables(wi_paged* pc, int batch, const int32_t* ctx_len, const int32_t* new_len,
                    const int32_t* free_pages, const int32_t* n_free, int free_cap, int32_t* block_table,
                    int32_t* kv_len, int32_t* q_start, int32_t* slots, int32_t* positions, int n_tokens,
                    int32_t* n_free_out, void* stream);

/*
 * Norms and rotation of a step's queries and keys, and their way into the
 * cache, in one pass.  q [n_tokens][n_q_heads][128], k and v
 * [n_tokens][n_kv_heads][128]: device bf16, heads contiguous, tokens
 * q_stride, k_stride, v_stride elements apart (multiples of 8; a fused
 * projection's rows can be passed as they are), 16-byte aligned.  Per head of
 * q and k: x * rsqrt(mean(x^2) + eps) * weight with q_weight / k_weight device
 * bf16 [128] (NULL: no norm), then each pair (a, b) of the rotated part by the
 * angle positions[t] * inv_freq[i]: (a cos - b sin, b cos + a sin).  All in
 * fp32, rounded once; the angle (in half a turn either way) is off by at most
 * 2^-31 of a turn and 2^-24 of itself, at any position.
 * Queries go to q_out [n_tokens][n_q_heads][128] (q itself if
 * q_stride = n_q_heads * 128; outputs share no memory otherwise, WI_EINVAL),
 * keys and values to slot slots[t] of the pools.
 * A token with positions[t] < 0 is padding: nothing of it is written; one with
 * slots[t] < 0 has its query written only.  Live tokens' slots are distinct.
 * With slots NULL, k_pages and v_pages are [n_tokens][n_kv_heads][128] instead
 * of pools: the layout of wi_decode_step's k_new and v_new (one layer).
 */
int wi_paged_write(wi_paged* pc, int n_tokens, const void* q, long long q_stride, const void* k, long long k_stride,
                   const void* v, long long v_stride, const void* q_weight, const void* k_weight,
                   const int32_t* positions, const int32_t* slots, void* q_out, void* k_pages, void* v_pages,
                   void* stream);

/*
 * Attention of a step's tokens over the cache (their own keys and values
 * already written).  q: device bf16 [n_tokens][n_q_heads][128], normed and
 * rotated; q_start [batch + 1] and kv_len [batch] as wi_paged_tables writes
 * them: where an entry of q_start lies below the one before it, the request that ends there and all behind it have no
 * tokens (and an error bit is set).  Token i of request b sits at position kv_len[b] - (tokens of b) + i
 * and sees positions 0 .. its own: out = softmax(q K^T / sqrt(128)) V, bf16
 * [n_tokens][n_q_heads][128]; lse (fp32 [n_tokens][n_q_heads], may be NULL)
 * the natural logarithm of the row's sum of exponentials.  A token whose
 * position is negative (kv_len smaller than the request's tokens) sees
 * nothing: out 0, lse -infinity.  Rows at and behind q_start[batch] stay as
 * they were.  What lies in the pools beyond a request's kv_len, or at
 * positions that a token does not see, has no influence, not even infinities
 * or NaN.  Fp32 accumulation (the tensor cores' over 2^18 positions at most,
 * then added up in turn) and softmax; the weights are rounded to bf16 for
 * the product with V (the row's sum is of the unrounded ones).  Same inputs,
 * same bits.  Single tokens and chunks may be mixed freely in one call.
 */
int wi_paged_attention(wi_paged* pc, int batch, int n_tokens, const void* q, const void* k_pages,
                       const void* v_pages, const int32_t* block_table, const int32_t* q_start,
                       const int32_t* kv_len, void* out, float* lse, void* stream);

/*
 * Rows out of the cache: positions [pos0, pos0 + n) of every request and of
 * `layers` consecutive pools (layer l's pools start l * n_pages * n_kv_heads *
 * page_size * 128 elements into k_pages / v_pages), to k_out and v_out: device
 * bf16 [batch][layers][n_kv_heads][n][128], as wi_build_index takes them, and with n = 1
 * wi_decode_step's k_new and v_new.  Positions at or beyond kv_len[b] become zeros.
 * layers <= 65536 (WI_EINVAL), batch * layers * n_kv_heads * n < 2^37.
 */
int wi_paged_gather(wi_paged* pc, int batch, int layers, const void* k_pages, const void* v_pages,
                    const int32_t* block_table, const int32_t* kv_len, long long pos0, long long n, void* k_out,
                    void* v_out, void* stream);

/*
 * The paged cache in 8 bits: half the memory, and half of what attention reads.
 * k_pages and v_pages are e4m3 [n_pages][n_kv_heads][page_size][128] (sign, 4
 * exponent bits of bias 7, 3 mantissa bits; largest 448; all ones is NaN, there
 * is no infinity), k_scales and v_scales [n_pages][n_kv_heads][page_size / 16]
 * bytes, one for every group of sixteen positions of a head: byte x is the factor
 * 2^(x - 127) on the group's values.  Device, the pools 16-byte aligned; tables,
 * lengths and slots are those of the bf16 pools.
 *
 * wi_paged_write8 is wi_paged_write into such pools (slots are needed).  What a
 * slot gets is the fp32 key or value over its group's scale, rounded to the
 * nearest e4m3 (ties to even; infinities and NaN become NaN).  A group's scale is
 * the smallest power of two, 2^-64 at least, with which its largest finite value
 * is 448 at most; so no value saturates, and a value keeps four significant bits
 * unless it is below 2^-6 of the scale.  It is worked out from what the call
 * writes and, where the call's first slot of the group is not the group's first,
 * from the scale that stands there: where that is larger it stays, else the rows
 * in front of the call's are rounded again to the new one, which loses nothing
 * but what falls below 2^-6 of it.  A group whose first slot the call writes
 * begins anew; rows behind the call's last stay as they were.  Tokens of one
 * call that share a group have to follow one another, in rising slots without a
 * gap (as wi_paged_tables gives them): otherwise that group's contents are
 * unspecified.
 * Unlike wi_paged_write, which touches the call's slots alone, a call may so
 * change values and scales that earlier ones wrote (of a group that it adds to,
 * the values in front of its own first, then the scale): what reads that group,
 * as attention or a gather of the same request, has to be ordered before the
 * call or behind it, on other streams with an event.
 */
int wi_paged_write8(wi_paged* pc, int n_tokens, const void* q, long long q_stride, const void* k, long long k_stride,
                    const void* v, long long v_stride, const void* q_weight, const void* k_weight,
                    const int32_t* positions, const int32_t* slots, void* q_out, void* k_pages, void* v_pages,
                    void* k_scales, void* v_scales, void* stream);

/*
 * wi_paged_attention over 8-bit pools: the same tables, rows and masks, with keys and values that are a pool's
 * values times their group's scale.  What lies at positions that a token does not see has no influence, NaN and
 * scales included.  Queries and weights are not rounded to 8 bits: a query's elements are held to 2^-17 of the largest
 * of their head (bf16's own bits down to 2^-9 of it); a weight, for the product with V, to 2^-11 of itself or to 2^-29
 * of the row's largest, whichever is more (2^-33 in calls of single tokens; where values' scales differ, weights times
 * scales are meant, and scales of 2^-64 or more).  The sum over the positions is an fp32 one whose additions cut bits
 * off: over many positions of values of one sign it comes out up to 2^-10 of itself too small (2^-16 in calls of single
 * tokens).  lse and the sum that divides have every weight down to 2^-30 of the largest in fp32, as long as the scales
 * of the values that a row sees lie within 2^100 of each other.
 * A call of no more tokens than requests (n_q_heads / n_kv_heads = 2: twice, 1: four times as many) is one of single
 * tokens: how the requests share the tokens does not change what it gives, but a chunk reads its context once for every
 * token (two, four) there.  Requests without tokens are better left out of a call that has a chunk.
 */
int wi_paged_attention8(wi_paged* pc, int batch, int n_tokens, const void* q, const void* k_pages,
                        const void* v_pages, const void* k_scales, const void* v_scales, const int32_t* block_table,
                        const int32_t* q_start, const int32_t* kv_len, void* out, float* lse, void* stream);

/*
 * wi_paged_gather from 8-bit pools: k_out and v_out are bf16, value times scale (exact, unless it leaves bf16's range).
 * Layer l's scales start l * n_pages * n_kv_heads * page_size / 16 bytes into k_scales / v_scales.
 */
int wi_paged_gather8(wi_paged* pc, int batch, int layers, const void* k_pages, const void* v_pages,
                     const void* k_scales, const void* v_scales, const int32_t* block_table, const int32_t* kv_len,
                     long long pos0, long long n, void* k_out, void* v_out, void* stream);

/* Error-path testing: with the environment variable WI_FAIL_ALLOC_AT=n (n >= 1),
 * the n-th device allocation made for any index fails as out-of-memory; the
 * call returns WI_ENOMEM having released what it had allocated.  Likewise
 * WI_FAIL_TIER_ALLOC_AT=n for the n-th allocation (device or page-locked
 * host) of wi_tier_attach, which then leaves the index as it was. */

/* Release the index and everything it owns (not k / v).  NULL is a no-op.
 * Synchronises the device first. */
void wi_free(wi_index* ix);

/* Message of the last failed call on this thread ("" if none). */
const char* wi_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* WAVE_INDEX_H */
