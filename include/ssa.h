/*
 * ssa.h -- C ABI of the GB300 (sm_103a) sparse-attention decode library.
 *
 * One decode step of one sparse-attention layer, for a batch of requests:
 *
 *   ssa_index_topk          int8 indexer over a compressed per-page key slab,
 *                           then a fixed-shape top-k page selection
 *   ssa_ensure_resident     device-side LRU: bind every selected logical page
 *                           to a physical GPU slot, fetch misses from the
 *                           pinned host mirror over UVA (NVLink-C2C)
 *   ssa_remap_block_table   selected logical pages -> physical slots
 *   ssa_sparse_paged_decode GQA decode attention over the selected pages only
 *
 * and the write path that fills the cache:
 *
 *   ssa_store_kv_mirror     quantise (8-bit formats) or pass through (bf16)
 *                           new K/V, write the pinned host mirror and, when
 *                           resident, the GPU slot; update the indexer slab
 *
 * and what a serving loop does around them:
 *
 *   ssa_rope, ssa_norm_rope rotary positions of queries and new keys, and the
 *                           norms of their heads in front
 *   ssa_prompt_attention    attention over whole prompts, on their way in
 *   ssa_beam_select         the next tokens of beams
 *   ssa_copy_pages, ssa_fork_requests, ssa_compact_pages
 *                           who owns the pages: copies, forks, growth, freed
 *                           requests, a compact page space
 *
 * Sources (web pages, cited by title and section):
 *   FreeToken PR #499 "host-RAM KV tier for sparse-attention models
 *     (--kv-host-pages)": "What", "Why this works for sparse attention",
 *     "Design", "Known limitations".
 *   FreeToken PR #525 "host-resident prefix tier for hybrid GDN models",
 *     conversation summary: mirror_store_quant, scale banks, select width.
 *   vLLM issue #33980 "[RFC]: Sparse attention KV cache offloading",
 *     "Motivation" and "Proposed Change".
 *
 * ---------------------------------------------------------------------------
 * Conventions for every call
 *   * Ownership: the caller allocates and owns every buffer.  Device buffers
 *     are plain device pointers; the host mirror is pinned host memory that
 *     the GPU can address (cudaHostAlloc / pinned torch tensors; on a
 *     unified-addressing system the host pointer is also the device pointer).
 *     The library allocates nothing and keeps no pointer after a call returns.
 *   * Streams: every call only enqueues work on `stream` (a cudaStream_t) and
 *     never synchronises the host, so a sequence of calls can be captured in
 *     a CUDA graph.  Calls on one stream are ordered; the caller orders
 *     streams.
 *   * Layers: every call takes a layer range [layer0, layer0 + n_layers).
 *     Cache arrays (ssa_cache) are indexed by absolute layer; per-call arrays
 *     (q, sel, phys, out, ...) hold n_layers consecutive layer slices, slice 0
 *     being layer0.  One launch covers the whole range.
 *   * Return value: SSA_OK, or a negative SSA_ERR_* found on the host before
 *     anything was enqueued (SSA_ERR_CUDA: a launch failed; the cudaError_t
 *     is kept for ssa_last_cuda_error()).
 *   * Device-detected problems set bits (atomicOr) in the caller's int32
 *     status word `status` (device memory, may be NULL): SSA_ST_*.  The word
 *     is never cleared by the library; the caller reads it when it chooses.
 *   * No kernel traps, asserts or waits without a bound: a wait that runs out
 *     sets SSA_ST_TIMEOUT and the kernel returns.
 * ---------------------------------------------------------------------------
 */
#ifndef SSA_H
#define SSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ABI-compatible with cudaStream_t. */
typedef struct CUstream_st *ssa_stream_t;

enum {
  SSA_OK = 0,
  SSA_ERR_INVALID_ARG = -1,   /* null pointer, bad range, bad layout field   */
  SSA_ERR_POOL_TOO_SMALL = -2,/* pool_slots < min(batch*max_sel, logical)    */
  SSA_ERR_UNSUPPORTED = -3,   /* dtype, page size, head_dim, GQA group       */
  SSA_ERR_NO_MIRROR = -4,     /* a host tier call without mirror pointers    */
  SSA_ERR_CUDA = -5,          /* a CUDA launch or attribute query failed     */
  SSA_ERR_SCRATCH_LIMIT = -6  /* ssa_index_topk_static_scratch: the call needs
                                 more than SSA_STATIC_SCORE_ENTRIES scores     */
};

enum {
  SSA_ST_DROP = 1,            /* a selection did not fit max_sel (counted)   */
  SSA_ST_BAD_ID = 2,          /* logical page id or page index out of range  */
  SSA_ST_MISS_NO_MIRROR = 4,  /* a miss had no host mirror to fetch from     */
  SSA_ST_UNRESOLVED = 8,      /* a selected page had no slot at remap/decode */
  SSA_ST_BAD_POS = 16,        /* store positions not strictly increasing     */
  SSA_ST_TIMEOUT = 32,        /* a bounded device wait gave up               */
  SSA_ST_INTERNAL = 64,       /* a kernel's own consistency check failed (its
                                 work was abandoned; report it as a bug)       */
  SSA_ST_NO_PAGES = 128       /* ssa_fork_requests found too few free pages    */
};

/* KV formats.  FP8_E4M3: e4m3 codes, one fp32 scale per token (over all KV
 * heads) for K and one for V.  The PAGE_HEAD formats: e4m3 or int8 codes, one
 * fp32 scale per page and KV head for K and one for V. */
enum {
  SSA_KV_BF16 = 0,
  SSA_KV_FP8_E4M3 = 1,
  SSA_KV_E4M3_PAGE_HEAD = 2,
  SSA_KV_INT8_PAGE_HEAD = 3
};

/*
 * Shapes.  Validated by every call.
 *   page_size   P, tokens per page: 16, 32, 64 or 128
 *   n_q_heads   Hq;  n_kv_heads Hkv;  G = Hq / Hkv must be an integer, 1..8
 *   head_dim    D, must be 128
 *   kv_dtype    one of SSA_KV_*
 *   n_layers    layers held by the cache arrays
 *   logical_pages  Lp, logical page ids per layer (0 .. Lp-1)
 *   pool_slots  S, physical GPU slots per layer
 *   batch       B requests;  max_pages n_max = block-table width
 *   block_topk  k >= 1;  max_sel W must equal 2*k + 8 (FreeToken PR #499,
 *               "Design": max_sel_pages sized from 2*block_topk + 8)
 */
typedef struct ssa_layout {
  int page_size, n_q_heads, n_kv_heads, head_dim;
  int kv_dtype;
  int n_layers, logical_pages, pool_slots;
  int batch, max_pages, block_topk, max_sel;
} ssa_layout;

/*
 * The paged KV cache and its residency state (all per layer, layer-major).
 *
 *   k_pool   [Lyr][S][Hkv][P][D]   bf16 values, or 8-bit codes
 *   v_pool   bf16: [Lyr][S][Hkv][P][D];  8-bit: [Lyr][S][Hkv][D][P] (each KV
 *            head's page stored d-major, tokens contiguous, so the attention
 *            kernel reads 8-bit V with tokens along the reduction)
 *   k_scale, v_scale   [Lyr][S][P] fp32 per-token scales (FP8_E4M3), or
 *            [Lyr][S][Hkv] fp32 scales of each page and KV head (PAGE_HEAD
 *            formats); NULL for bf16
 *   k_mirror, v_mirror, k_scale_mirror, v_scale_mirror: the same per-page
 *            blocks indexed by logical page, [Lyr][Lp][...], in pinned host
 *            memory; all four NULL means no host tier.  Mirror bytes equal
 *            pool bytes for every bound slot (FreeToken PR #525: the mirror
 *            holds the codes and scales after quantisation).
 *   slab       [Lyr][Lp][Hkv][D] int8 page-mean key codes (the indexer slab)
 *   slab_scale [Lyr][Lp] fp32, the per-page symmetric scale amax/127
 *   slab_sum   [Lyr][Lp][Hkv][D] fp32 running key sums (token order)
 *   slab_cnt   [Lyr][Lp] int32 tokens summed
 *   slot_of  [Lyr][Lp]  physical slot of a logical page, or -1
 *   page_of  [Lyr][S]   logical page held by a slot, or -1 (free)
 *   last_use [Lyr][S]   clock value of the slot's last use, -1 never
 *   clock    [Lyr]      ensure steps taken
 * Device pointers except the mirrors.  All 256-byte aligned, except that
 * scale arrays need 16 bytes.
 */
typedef struct ssa_cache {
  void *k_pool, *v_pool;
  float *k_scale, *v_scale;
  void *k_mirror, *v_mirror;
  float *k_scale_mirror, *v_scale_mirror;
  int8_t *slab;
  float *slab_scale;
  float *slab_sum;
  int32_t *slab_cnt;
  int32_t *slot_of, *page_of, *last_use, *clock;
} ssa_cache;

/* Bytes of scratch (device memory, 256-byte aligned) that ssa_index_topk,
 * ssa_ensure_resident, ssa_sparse_paged_decode and the page calls need for any
 * layer range of this layout.  The calls use disjoint parts of it (the page
 * calls one part together).  Zero the workspace
 * once before its first use: ssa_sparse_paged_decode keeps per-unit split
 * counters in it, ssa_fork_requests a ticket and marks, and every call that
 * completes leaves them zero again (a call that reported SSA_ST_TIMEOUT may
 * not: zero the workspace again).
 * 0 on a bad layout. */
size_t ssa_workspace_size(const ssa_layout *lay);

/*
 * Reset the residency state of every layer (FreeToken PR #499, "What": the
 * GPU's slots cache logical pages, least recently used out first).
 *   identity = 0: empty pool (slot_of = page_of = last_use = -1, clock 0);
 *   identity = 1: fully resident, slot s holds logical page s for
 *                 s < min(S, Lp), last_use -1, clock 0.
 * Also zeroes slab, slab_scale, slab_sum and slab_cnt.
 */
int ssa_lru_init(const ssa_layout *lay, const ssa_cache *c, int identity,
                 ssa_stream_t stream);

/*
 * a0 -- store K/V through the write-through mirror (FreeToken PR #499,
 * "Design": each stored token also goes to pinned host memory, so evicting a
 * slot never needs a write-back; FreeToken PR #525: with fp8 the host copy
 * holds the quantised codes and their scales, byte for byte the pool's).
 *   k, v   [n_layers][T][Hkv][D] bf16, device
 *   pos    [T] int64 logical token ids, page = pos / P, row j = pos % P;
 *          strictly increasing within the call (SSA_ST_BAD_POS otherwise),
 *          each position stored once over the cache's lifetime
 * A call holds any run of tokens: a prefill chunk, or the one token per
 * request a decode step appends; a page may be filled over many calls, and
 * its slab row then equals that of one call storing the same tokens.
 * fp8: per token and tensor, s = max|x| / 448 over all KV heads (1 if the
 * token is all zero), code = e4m3(x / s) rounded to nearest even,
 * saturating.  Writes the mirror always (when present) and the pool slot
 * when the page is resident.  Slab: adds each token's bf16 keys to slab_sum
 * in token order, counts them, and re-quantises the touched pages:
 * mean = sum / count, s = max|mean| / 127, code = clamp(rint(mean/s), +-127)
 * (all zero when max|mean| = 0).  Out-of-range pages: SSA_ST_BAD_ID.
 *
 * PAGE_HEAD formats: per page, KV head and tensor, with amax the largest
 * finite |x| of the call's tokens of that page and qmax = 448 (e4m3) or 127
 * (int8):
 *   need = amax / qmax;  s' = need on a page without tokens (slab_cnt 0),
 *   else max(s, need);
 *   when s' > s on a page with tokens, every code of the block becomes
 *   Q(code * (s / s'));
 *   the new codes are Q(x / s'), all zero when s' = 0,
 * with Q rounding to nearest even (int8 clamped to +-127, NaN -> 0; e4m3
 * saturating).  So a page's scale only grows, and pages filled over several
 * calls can hold codes that were rounded more than once (at most half a code
 * step each time the scale grew).  k and v must be 16-byte aligned.
 */
int ssa_store_kv_mirror(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                        const void *k, const void *v, const int64_t *pos, int T,
                        int32_t *status, ssa_stream_t stream);

/*
 * a1 + a2 -- indexer and top-k page selection (FreeToken PR #499, "Why this
 * works for sparse attention": every attend step first runs top-k block
 * selection over the compressed, GPU-resident slab, fixed shape; "Design":
 * compact_selected_pages with a drop counter).
 *   q           [n_layers][B][Hq][D] bf16, device
 *   block_table [B][n_max] int32 logical page ids of each request's pages
 *   seq_lens    [B] int32 tokens per request; n_b = ceil(seq_len / P) pages
 *   sel         [n_layers][B][W] int32 out: selected page indices (into the
 *               request's block-table row), ascending, -1 padded
 *   n_sel       [n_layers][B] int32 out
 *   scores_opt  [n_layers][B][n_max] int32 out or NULL; INT32_MIN past n_b
 * q is quantised per request: s = max|q| / 127 over all Hq*D values,
 * q8 = clamp(rint(q/s), +-127).  Score of page p (exact int32):
 *   S[p] = sum_hq sum_d q8[hq][d] * slab[bt[p]][hq / G][d].
 * Selection: the k best of pages [0, n_b - 1) by (score desc, page asc),
 * plus page n_b - 1 always; all pages when n_b - 1 <= k.  Selections that
 * would not fit W are dropped and flagged SSA_ST_DROP (cannot happen when
 * W = 2k + 8).  One launch: the last CTA to finish scoring a (layer,
 * request) row selects over it.  ws: ssa_workspace_size bytes, zeroed once
 * (required; it holds the per-row tickets).
 */
int ssa_index_topk(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                   const void *q, const int32_t *block_table, const int32_t *seq_lens,
                   int32_t *sel, int32_t *n_sel, int32_t *scores_opt, int32_t *status,
                   void *ws, ssa_stream_t stream);

/*
 * a3 + a4 -- LRU ensure and miss fetch (FreeToken PR #499, "Design": the
 * LRU runs on the device with fixed shapes, so it can sit in a CUDA graph;
 * evicting only rebinds a slot; misses are copied host -> device; FreeToken
 * PR #525: the copy includes the fp8 scales, and the pool is sized so that
 * the whole batch's selection fits).
 * Per layer, in this order:
 *   1. U = distinct logical ids bt[b][sel[b][i]] of the batch, ascending;
 *   2. hits are touched: last_use[slot] = clock;
 *   3. misses (ascending id) take victims in order: free slots by ascending
 *      slot id, then bound slots not touched this step by ascending
 *      (last_use, slot); the victim's old page loses its slot;
 *   4. each miss's K, V (and fp8 scales) are copied mirror -> slot;
 *   5. clock += 1.
 *   sel                    [n_layers][B][W] from ssa_index_topk
 *   miss_page_opt, miss_slot_opt  [n_layers][B*W] int32 out or NULL
 *   n_miss_opt             [n_layers] int32 out or NULL
 * Requires pool_slots >= min(B*W, Lp) (SSA_ERR_POOL_TOO_SMALL).  A miss
 * without a mirror is bound but not fetched: SSA_ST_MISS_NO_MIRROR.
 */
int ssa_ensure_resident(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                        const int32_t *sel, const int32_t *block_table,
                        int32_t *miss_page_opt, int32_t *miss_slot_opt, int32_t *n_miss_opt,
                        int32_t *status, void *ws, ssa_stream_t stream);

/*
 * a3 + a4 + a5 in one call: ssa_ensure_resident, whose LRU kernel also
 * writes the remapped table once every selected page has its slot -- the
 * same phys as ssa_remap_block_table (FreeToken PR #499, "Design": after
 * ensure the block table is translated logical -> physical), one launch
 * fewer per step.
 *   phys [n_layers][B][W] int32 out (required)
 */
int ssa_ensure_remap(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                     const int32_t *sel, const int32_t *block_table, int32_t *phys,
                     int32_t *miss_page_opt, int32_t *miss_slot_opt, int32_t *n_miss_opt,
                     int32_t *status, void *ws, ssa_stream_t stream);

/*
 * ssa_ensure_remap in two calls, so that the host-link copy of one layer
 * range can run while the attention of another range reads its pages
 * (vLLM RFC #33980, "Motivation": the load time is what has to be hidden;
 * FreeToken PR #499, "Design": ensure, then copy, then attend, per layer).
 *   ssa_ensure_remap_bind: steps 1-3 and 5 of ssa_ensure_resident and the
 *     remap of ssa_ensure_remap -- the residency state, phys and the miss
 *     lists are final -- but nothing is copied;
 *   ssa_fetch_misses: step 4 for the layers [layer0, layer0 + n_layers):
 *     each listed miss's K, V (and fp8 scales) mirror -> slot.  Any split of
 *     a bind call's range into fetch calls (lists offset to the first layer
 *     of each) gives the bytes of the one ssa_ensure_remap call.
 * Between the two, a missed page's slot holds stale bytes while phys already
 * names it: the attention over a layer goes after that layer's fetch (same
 * stream, or an event), and no other call on those layers goes between.
 *   phys           [n_layers][B][W] int32 out (bind)
 *   miss_page, miss_slot  [n_layers][B*W] int32, out (bind) / in (fetch)
 *   n_miss         [n_layers] int32, out (bind) / in (fetch)
 * The lists are required (no workspace default).  The fetch needs the host
 * mirror (SSA_ERR_NO_MIRROR); the bind flags a miss without one on the
 * device, as ssa_ensure_resident does.
 */
int ssa_ensure_remap_bind(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                          const int32_t *sel, const int32_t *block_table, int32_t *phys,
                          int32_t *miss_page, int32_t *miss_slot, int32_t *n_miss,
                          int32_t *status, ssa_stream_t stream);
int ssa_fetch_misses(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                     const int32_t *miss_page, const int32_t *miss_slot, const int32_t *n_miss,
                     int32_t *status, ssa_stream_t stream);

/*
 * The miss fetch folded into the attention: ssa_ensure_remap_deferred runs
 * the ensure's state update and remap (a3, a5) but copies nothing; its phys
 * marks each page this call bound (a miss) as -2 - slot.  Then
 * ssa_sparse_paged_decode_fetch runs the attention on that phys: a marked
 * page is read from the pinned host mirror inside the attention kernel (the
 * host-tail path), used, and written into its slot as it streams past, so
 * the host-link reads overlap the attention over the resident pages instead
 * of preceding it (FreeToken PR #499, "Design": ensure, then copy, then
 * attend; vLLM RFC #33980, "Motivation": the load time is what has to be
 * hidden).  The residency state, the miss lists, the pool bytes afterwards
 * and the outputs are those of ssa_ensure_remap + ssa_sparse_paged_decode.
 * Between the two calls the marked slots hold stale bytes: nothing else may
 * read them, and the pair must not be split across other calls on the
 * cache.  Both require the host mirror (SSA_ERR_NO_MIRROR).
 *   phys [n_layers][B][W] int32 out / in: slot, -2 - slot (marked), or -1
 *   block_table (fetch): as for ssa_index_topk, for the marked pages' ids
 */
int ssa_ensure_remap_deferred(const ssa_layout *lay, const ssa_cache *c, int layer0,
                              int n_layers, const int32_t *sel, const int32_t *block_table,
                              int32_t *phys, int32_t *miss_page_opt, int32_t *miss_slot_opt,
                              int32_t *n_miss_opt, int32_t *status, void *ws,
                              ssa_stream_t stream);
int ssa_sparse_paged_decode_fetch(const ssa_layout *lay, const ssa_cache *c, int layer0,
                                  int n_layers, const void *q, const int32_t *sel,
                                  const int32_t *phys, const int32_t *block_table,
                                  const int32_t *seq_lens, float sm_scale, void *out,
                                  int32_t *status, void *ws, ssa_stream_t stream);

/*
 * Residency shared by the layers of a call (FreeToken PR #499, "Design": one
 * launch copies a page's K and V for all the sparse-attention layers).  The
 * layers [layer0, layer0 + n_layers) share ONE LRU state, layer0's slot_of /
 * page_of / last_use / clock (the other layers' state arrays are not used):
 *   1. U = distinct logical ids selected by any layer of the range, ascending;
 *   2-5. as ssa_ensure_resident, on that one state: hits touched, misses take
 *      free slots then untouched slots by (last_use, slot), rebind, clock + 1;
 *      each miss's K, V (and scales) are copied into the same slot of
 *      EVERY layer's pool (one launch for all layers);
 *   then phys [n_layers][B][W] = slot_of[layer0][bt[b][sel]] for every layer.
 *   miss_page_opt, miss_slot_opt [n_layers * B * W] int32 out or NULL
 *   n_miss_opt  [1] int32 out or NULL: misses of the call
 * Requires n_layers * B * W <= 16384 (SSA_ERR_UNSUPPORTED) and pool_slots >=
 * min(n_layers * B * W, logical_pages) (SSA_ERR_POOL_TOO_SMALL).  Use one
 * residency mode per cache: this call and ssa_ensure_resident / ssa_ensure_remap
 * keep different state.  ssa_store_kv_mirror goes by each layer's own slot_of:
 * for a store that may touch pages that hold a slot, copy layer0's row over the
 * other layers' and set those back to -1 after the call.
 */
int ssa_ensure_remap_shared(const ssa_layout *lay, const ssa_cache *c, int layer0,
                            int n_layers, const int32_t *sel, const int32_t *block_table,
                            int32_t *phys, int32_t *miss_page_opt, int32_t *miss_slot_opt,
                            int32_t *n_miss_opt, int32_t *status, void *ws,
                            ssa_stream_t stream);

/*
 * Top-k preload (vLLM RFC #33980, "Motivation" point 2 and "Proposed Change":
 * "Topk KV preload" -- adjacent decode steps select largely the same pages,
 * so a former top-k can drive a fetch that overlaps the current step's
 * compute, leaving only the residual misses to load once the actual top-k
 * is known).  Run after a step's ssa_ensure_resident, on that step's scores:
 *   1. candidates, per request: the top (width - 1) pages of [0, n_b - 1) by
 *      (score desc, page asc) plus page n_b - 1 (all pages when
 *      n_b - 1 <= width - 1) -- the selection rule with k = width - 1;
 *   2. per layer, U = the distinct logical ids of the batch's candidates;
 *      with e = clock - 1 (the epoch of the step's ensure):
 *   3. resident ids of U are touched: last_use = e;
 *   4. the other ids of U, ascending, take victims in order: free slots by
 *      ascending slot id, then bound slots with last_use < e by ascending
 *      (last_use, slot) -- so the pages the step's attention reads are never
 *      evicted; ids left over when no victim remains are not fetched;
 *   5. each bound id gets last_use = e and its K, V (and fp8 scales) are
 *      copied mirror -> slot; the clock is not advanced.
 * The next ssa_ensure_resident then finds the fetched pages resident.
 *   scores        [n_layers][B][n_max] int32: the step's scores_opt from
 *                 ssa_index_topk; must not change until this call completes
 *   width         candidates per request, 1 <= width <= max_sel
 *   fetch_page_opt, fetch_slot_opt  [n_layers][B*W] int32 out or NULL
 *   n_fetch_opt   [n_layers] int32 out or NULL: pages fetched per layer
 * ws is required (the candidates and fetch lists live in a part of it that
 * no other call uses).  Ordering: after the step's ssa_remap_block_table
 * (which reads the state this call changes) and before the next step's
 * ssa_ensure_resident; it may run on a second stream concurrently with the
 * step's ssa_sparse_paged_decode (the slots it reads are never victims) and
 * the next step's ssa_index_topk (which must write its scores elsewhere).
 * SSA_ERR_POOL_TOO_SMALL as ssa_ensure_resident.
 */
int ssa_prefetch_pages(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                       const int32_t *scores, const int32_t *block_table,
                       const int32_t *seq_lens, int width, int32_t *fetch_page_opt,
                       int32_t *fetch_slot_opt, int32_t *n_fetch_opt, int32_t *status, void *ws,
                       ssa_stream_t stream);

/*
 * a5 -- block-table translation (FreeToken PR #499, "Design": after ensure
 * the block table is translated logical -> physical and attention runs on
 * it unmodified).
 *   phys [n_layers][B][W] int32 out: slot_of[bt[b][sel]] or -1 for padding;
 *   a selected page without a slot gives -1 and SSA_ST_UNRESOLVED.
 */
int ssa_remap_block_table(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                          const int32_t *sel, const int32_t *block_table, int32_t *phys,
                          int32_t *status, ssa_stream_t stream);

/*
 * a6 + a7 -- paged GQA decode attention over the selected pages only
 * (FreeToken PR #499, "Design": qsa_sparse_paged_attention runs on the
 * remapped table).  For request b and query head hq (KV head h = hq / G):
 *   out[b][hq] = sum_t softmax_t(sm_scale * q[b][hq] . K[t]) V[t]
 * over tokens t = p*P + j of the pages p = sel[b][i] with phys[b][i] >= 0
 * and t < seq_lens[b]; K[t] = code * k_scale[t] for fp8, code *
 * k_scale[slot][h] for the PAGE_HEAD formats (V likewise).
 * Entries with sel < 0 are padding; sel >= 0 with phys < 0 are skipped and
 * flagged SSA_ST_UNRESOLVED.  A request with no token gets zeros.
 *   q    [n_layers][B][Hq][D] bf16;  out [n_layers][B][Hq][D] bf16
 * One wave of CTAs cuts the (layer, request, KV head) x page work into equal
 * ranges (each (layer, request, KV head) weighs min(max_pages, block_topk+1)
 * pages, the selection size of a request with at least block_topk + 1
 * pages); a (layer, request, KV head) split between CTAs is merged by the
 * last of its pieces to finish, found by an atomic ticket.  ws is required:
 * it holds the partial softmax states and the tickets (zeroed before first
 * use, left zero by every call that completes).  SSA_ERR_INVALID_ARG when
 * ws is NULL.
 */
int ssa_sparse_paged_decode(const ssa_layout *lay, const ssa_cache *c, int layer0, int n_layers,
                            const void *q, const int32_t *sel, const int32_t *phys,
                            const int32_t *seq_lens, float sm_scale, void *out,
                            int32_t *status, void *ws, ssa_stream_t stream);

/*
 * Zero-copy host-tail attention (vLLM RFC #33980, the comment that maps one
 * address range with an HBM-backed head and a host-backed tail, so that the
 * attention reads the tail's slots over the interconnect with no staging
 * copy).  The same attention as ssa_sparse_paged_decode, on sel and the
 * block table instead of a remapped table: each selected page is resolved
 * through slot_of; a resident page is read from its pool slot, a page with
 * no slot straight from the pinned host mirror (16-byte loads over UVA into
 * the same on-chip layout).  The residency state is not changed -- no
 * ensure, no copy, no eviction -- so each step re-reads its host pages.
 *   sel          [n_layers][B][W] from ssa_index_topk
 *   block_table  [B][n_max] logical ids
 * Requires the host mirror (SSA_ERR_NO_MIRROR); ws as for
 * ssa_sparse_paged_decode.  Mirror bytes equal pool bytes, so the result is
 * that of ensure + remap + ssa_sparse_paged_decode on the same selection.
 */
int ssa_sparse_paged_decode_host_tail(const ssa_layout *lay, const ssa_cache *c, int layer0,
                                      int n_layers, const void *q, const int32_t *sel,
                                      const int32_t *block_table, const int32_t *seq_lens,
                                      float sm_scale, void *out, int32_t *status, void *ws,
                                      ssa_stream_t stream);

/*
 * Owners of the pages: copying pages, forking, growing and freeing requests,
 * compacting the logical page space.  (FreeToken PR #499, "What", has logical
 * pages that outlive the requests that filled them; the pages leave handing
 * them out to the engine around the cache.)
 *   block_table [B][n_max], seq_lens [B]: as for ssa_index_topk, here updated
 *   ref [Lp]  references of each logical page, device: one per row and entry
 *             below ceil(seq_len / P), plus any the caller adds to pin a page
 *             (a cached prefix, say).  ref <= 0: the page is free.
 * The calls work on every layer of the cache.  They order like every other
 * call; between ssa_ensure_remap_bind / _deferred and the call that completes
 * it none of them may run, and work on other streams (a preload) must have
 * been waited for.  ws: ssa_workspace_size bytes, zeroed once, not used by
 * another call at the same time.  With residency shared by the layers
 * (ssa_ensure_remap_shared) the other layers' state arrays must be unbound, as
 * ssa_lru_init leaves them, and a page that holds a slot is no dst of
 * ssa_copy_pages (only layer0's pool block would be written).  Lengths outside [0, n_max * P] set
 * SSA_ST_BAD_POS and count as the nearest bound; ids out of range set
 * SSA_ST_BAD_ID and are carried along, never followed.
 */
typedef struct ssa_requests {
  int32_t *block_table, *seq_lens, *ref;
} ssa_requests;

/* ref := the references of the table's rows (any pins are forgotten). */
int ssa_page_refs(const ssa_layout *lay, const ssa_requests *r, int32_t *status,
                  ssa_stream_t stream);

/*
 * Page dst[i] := page src[i], in every layer: K, V and scales, in the mirror
 * (where there is one) and in the slot that dst[i] holds (if any), and the
 * slab row.  The source is src[i]'s slot, or its mirror block.
 *   src, dst  [n] int32 device; n <= 16384 (SSA_ERR_UNSUPPORTED above);
 *             a pair with a negative id is padding
 * Pairs with an id out of range, whose dst is the dst of an earlier pair, or
 * the src of another pair, are skipped: SSA_ST_BAD_ID.  Without a mirror, a
 * page without a slot has no K and V to copy (SSA_ST_UNRESOLVED; the slab row
 * is copied).  Reference counts and residency stay as they are.
 */
int ssa_copy_pages(const ssa_layout *lay, const ssa_cache *c, const int32_t *src,
                   const int32_t *dst, int n, int32_t *status, void *ws, ssa_stream_t stream);

/*
 * Fork, grow and free requests: row i becomes a continuation of what row
 * parent[i] held before the call, max(its length, new_lens[i]) tokens long.
 *   parent[i] = i    the row goes on (and may grow)
 *   parent[i] = j    the row's own pages are let go; it shares j's context
 *   parent[i] = -1   the row is freed (new_lens[i] > 0: and admitted anew,
 *                    with new_lens[i] tokens' worth of empty pages)
 *   parent [B] int32, new_lens_opt [B] int32 or NULL (no growth); device
 * Full pages are shared.  A partly filled last page is kept by the lowest row
 * that continues it, unless a reference from elsewhere stays (a row that holds
 * it as a full page, a pin); every other row gets a copy (as ssa_copy_pages).
 * New pages are the lowest free ids, in row order (the copy, then growth);
 * pages let go in this call count as free.  New pages start with an empty slab
 * row.  A page that a row goes on holding is never a new one: if nothing counts
 * it (the row's length grew past the page by other means than this call, after
 * the counting), it gets a count of one and SSA_ST_BAD_ID is set.
 * With a mirror, new pages and pages that became free give their slots
 * back; without one every page keeps the slot it has (so a cache without a
 * mirror wants pool_slots >= logical_pages: a new page without a slot holds no
 * K and V).  Entries past a row's pages become -1.
 * Too few free pages: SSA_ST_NO_PAGES, and the rows that got none are cut to
 * the tokens their pages hold (a missing copy cuts the partly filled page).
 * A parent below -1 or at B and above: SSA_ST_BAD_ID, the row goes on; a
 * new_lens above n_max * P: SSA_ST_BAD_POS, clipped.
 */
int ssa_fork_requests(const ssa_layout *lay, const ssa_cache *c, const ssa_requests *r,
                      const int32_t *parent, const int32_t *new_lens_opt, int32_t *status,
                      void *ws, ssa_stream_t stream);

/*
 * Compaction: with n live pages (ref > 0), every live page gets an id below n,
 * so that the ids from n on (and their mirror blocks) are free.  The k-th live
 * page at or above n moves to the k-th free id below n, both ascending: slab
 * row, mirror block and count move, the two pages trade their slots (pool
 * bytes stay), and the rows name the new id.
 *   moved_from_opt, moved_to_opt [Lp] int32 out or NULL: the first n_moved
 *   entries are the moves (for references that the caller keeps itself)
 *   n_moved_opt [1] int32 out or NULL
 * Row entries whose page nothing counts set SSA_ST_BAD_ID; their pages are free
 * to be moved onto, so count first (ssa_page_refs, ssa_fork_requests).
 */
int ssa_compact_pages(const ssa_layout *lay, const ssa_cache *c, const ssa_requests *r,
                      int32_t *moved_from_opt, int32_t *moved_to_opt, int32_t *n_moved_opt,
                      int32_t *status, void *ws, ssa_stream_t stream);

/*
 * Rotary positions of queries and keys, before ssa_store_kv_mirror (keys) and
 * ssa_index_topk / ssa_sparse_paged_decode (queries).  (The pages take q and
 * k as given; every model that fills such a cache rotates them first.)  Pair
 * i < rotary_dim / 2 of a head is (x[i], x[i + rotary_dim / 2]), or (x[2i],
 * x[2i + 1]) with `interleaved`; dimensions from rotary_dim on are copied.
 *   angle = (pos[t] + pos_offset) * theta_i,  (c, s) = factor (cos, sin)(angle)
 *   a' = a c - b s,  b' = b c + a s     (inverse: s -> -s, which is also the
 *                                        gradient of the rotation)
 *   dtype     SSA_BF16, SSA_F16 or SSA_F32; computed in fp32, rounded once
 *   freq      [rotary_dim / 2] device: theta_i / (2 pi) as a 64-bit fraction
 *             of a turn (ssa_rope_frequencies), so that the angle is exact
 *             modulo a turn at any position
 *   pos       [n_tokens] device, int32 or (pos_is_64) int64; may be negative
 *   q, k      at most one NULL: heads, and element strides of layer, token and
 *             head (elements of a head are contiguous), so that a slice of a
 *             fused projection needs no copy.  out == in (same strides) rotates
 *             in place; otherwise the two must not overlap.  What one of q
 *             and k writes must not overlap what the other reads or writes.
 * 16-byte accesses where pointers, strides and dimensions allow, single
 * elements otherwise; same values either way.
 */
enum { SSA_BF16 = 0, SSA_F16 = 1, SSA_F32 = 2 };
#define SSA_ROPE_MAX_DIM 1024
typedef struct ssa_rope_tensor {
  const void *in;
  void *out;
  int heads;
  int64_t in_stride[3], out_stride[3];   /* layer, token, head */
} ssa_rope_tensor;
int ssa_rope(int dtype, int head_dim, int rotary_dim, int interleaved, int inverse,
             const uint64_t *freq, float factor, int n_layers, int n_tokens, const void *pos,
             int pos_is_64, int64_t pos_offset, const ssa_rope_tensor *q,
             const ssa_rope_tensor *k, ssa_stream_t stream);

/*
 * Norms of queries and keys, head by head, and their rotary positions in one
 * pass (models that norm q and k do so right before the rotation):
 *   y = x / sqrt(mean(x^2) + eps) * w,  then ssa_rope's rotation of y
 * over the head_dim elements of every (layer, token, head); in fp32 (in whose
 * range the sum of squares must stay), rounded once.  Arguments as for ssa_rope (no inverse), and
 *   q_weight, k_weight  [n_layers][head_dim] fp32, device, weight_step floats
 *             from one layer's to the next's (0: all layers share them); NULL:
 *             ones
 *   eps       finite, not negative
 */
int ssa_norm_rope(int dtype, int head_dim, int rotary_dim, int interleaved, const uint64_t *freq,
                  float factor, int n_layers, int n_tokens, const void *pos, int pos_is_64,
                  int64_t pos_offset, const ssa_rope_tensor *q, const ssa_rope_tensor *k,
                  const float *q_weight, const float *k_weight, int64_t weight_step, float eps,
                  ssa_stream_t stream);

/*
 * The frequency table of ssa_rope, on the host: theta_i = base^(-2i /
 * rotary_dim), changed for contexts longer than the model was trained on:
 *   PLAIN   as it is
 *   LINEAR  theta / factor
 *   NTK     base * factor^(rotary_dim / (rotary_dim - 2)) in place of base
 *   BANDS   by the turns n = original_len * theta / (2 pi) a pair makes over
 *           the original length: theta / factor for n <= low, theta for
 *           n >= high, and linear in n between the two
 *   YARN    theta / factor and theta blended along the pair index, from the
 *           pair that makes `high` turns over original_len (theta) to the one
 *           that makes `low` (theta / factor), both rounded outwards; the
 *           attention factor is 0.1 ln(factor) + 1 (1 for the others)
 *   freq         [rotary_dim / 2] out, host
 *   attn_factor  out or NULL: the `factor` argument of ssa_rope
 */
enum { SSA_ROPE_PLAIN = 0, SSA_ROPE_LINEAR = 1, SSA_ROPE_NTK = 2, SSA_ROPE_BANDS = 3,
       SSA_ROPE_YARN = 4 };
int ssa_rope_frequencies(int rotary_dim, double base, int scaling, double factor,
                         double original_len, double low, double high, uint64_t *freq,
                         double *attn_factor);

/*
 * Attention over whole prompts, on the way into the cache (the pages start from a
 * filled cache; a model's prompt attends over itself first).  Sequences of
 * different lengths lie one behind the other: sequence s has the query tokens
 * [cu_q[s], cu_q[s + 1]) of q and the keys [cu_kv[s], cu_kv[s + 1]) of k and v.
 * With Lq query tokens and Lk keys, query token i of a sequence and its head
 * hq = h * G + g, G = Hq / Hkv:
 *   out = sum_j w_j v_j[h],  w = softmax_j(sm_scale * q . k_j[h]),
 *   over j <= i + Lk - Lq (causal: the query tokens are the last ones of the
 *   keys' sequence, so keys that came before need not be passed as queries) or
 *   over all j < Lk
 *   lse = ln sum_j exp(sm_scale * q . k_j[h])
 * A query token that sees no key gets zeros and lse -inf; tokens outside every
 * sequence are left as they were.  What a row does not see has no part in it,
 * infinities and NaN among it.
 *   dtype     SSA_BF16 or SSA_F16, of q, k, v and out; scores, softmax and sums
 *             in fp32, weights rounded to dtype before they meet v and divided by
 *             the sum of the rounded ones (fp16 weights lose bits below 2^-21 of a
 *             row's greatest, and those below 2^-32 go)
 *   head_dim  128;  G at most 128
 *   q, out    [n_q][Hq][128];  k, v [n_kv][Hkv][128], 16-byte aligned; element
 *             strides of token and head, positive multiples of 8, so that
 *             slices of a fused projection need no copy.  No element of out is
 *             another's or twice in out; where it lies between the rows of an
 *             input, both have the same token stride (SSA_ERR_INVALID_ARG)
 *   cu_q, cu_kv  [n_seqs + 1] int32, device, ascending, within the tensors
 *             (SSA_ST_BAD_POS otherwise; nothing outside the tensors is read
 *             or written).  The same array where queries and keys are the same
 *             tokens.
 *   sm_scale  finite, not negative
 *   lse_opt   [n_q][Hq] fp32 out, or NULL
 *   ws        ssa_prompt_workspace_size() bytes, 16-byte aligned, not used by
 *             another call at the same time; needs no clearing
 * Where a call has few rows and many keys the keys are split over the machine
 * and the parts joined in a fixed order: the same inputs give the same bits.
 */
typedef struct ssa_prompt_tensor {
  void *data;
  int heads;
  int64_t stride[2];                     /* token, head */
} ssa_prompt_tensor;
size_t ssa_prompt_workspace_size(void);
int ssa_prompt_attention(int dtype, int head_dim, int n_seqs, int n_q, int n_kv,
                         const ssa_prompt_tensor *q, const ssa_prompt_tensor *k,
                         const ssa_prompt_tensor *v, const ssa_prompt_tensor *out,
                         const int32_t *cu_q, const int32_t *cu_kv, int causal, float sm_scale,
                         float *lse_opt, int32_t *status, void *ws, ssa_stream_t stream);

/*
 * The next tokens of beams, and what ssa_fork_requests needs to follow them
 * (which pages a beam goes on with; the pages leave the choice to the engine).
 * Groups of `beams` rows, rows g * beams .. of a batch, logits x[row][vocab]:
 *   a candidate (row, t) has the score  scores[row] + x[row][t] - ln sum_t' exp(x[row][t'])
 *   a finished row has one candidate, (row, eos), at scores[row]
 *   logits of -infinity and NaN (a mask) are no candidates, nor is anything of a
 *   row whose score is -infinity or NaN; logits above 2^126 count as 2^126
 * The `beams` best of each group, best first, equal scores by the lower row and
 * then the lower token, become the group's rows; the best of several rows may
 * be of one parent.  Sums in 64-bit integers (each exponential is off by about
 * 2^-22 of itself), scores in double, one rounding to fp32 at the end.
 *   dtype     SSA_BF16, SSA_F16 or SSA_F32, of the logits
 *   logits    [groups * beams] rows, row_stride elements apart
 *   groups at most 65,535, beams at most 32, vocab at most 2^23 (SSA_ERR_UNSUPPORTED)
 *   in, out   the rows' state before and after; out may be in:
 *     scores    [groups * beams] fp32 (a first step: 0 for one row of a group
 *               and -infinity for the others)
 *     finished  [groups * beams] bytes, with eos >= 0; NULL without (eos = -1)
 *     history   [groups * beams][max_len] int32, hist_len [groups] the tokens in
 *               a row of it; both NULL with max_len = 0.  Rows are reordered
 *               and the new token appended; where the row is full, or its
 *               length not in [0, max_len], the token is not kept and
 *               SSA_ST_BAD_POS set.  Nothing behind the new token is written.
 *   parent    [groups * beams] int32 out: the row (of the batch) each continues,
 *             -1 where the group has too few candidates: token -1, score
 *             -infinity, not finished, its history left as it was
 *   token     [groups * beams] int32 out
 *   seq_lens_opt, new_lens_opt  [groups * beams] int32, both or none:
 *             new_lens[row] = seq_lens[parent] + 1, 0 for parent -1, as
 *             ssa_fork_requests takes them (may be the same array).  That of a
 *             beam that has ended grows too, a token a call, as its history does
 *   ws        ssa_beam_workspace_size(groups, beams) bytes or more, 256-byte
 *             aligned, zeroed once, not used by another call at the same time;
 *             calls of any sizes that it is large enough for may take turns
 */
typedef struct ssa_beams {
  float *scores;
  uint8_t *finished;
  int32_t *history, *hist_len;
} ssa_beams;
size_t ssa_beam_workspace_size(int groups, int beams);
int ssa_beam_select(int dtype, int groups, int beams, int vocab, const void *logits,
                    int64_t row_stride, const ssa_beams *in, const ssa_beams *out, int max_len,
                    int eos, int32_t *parent, int32_t *token, const int32_t *seq_lens_opt,
                    int32_t *new_lens_opt, int32_t *status, void *ws, ssa_stream_t stream);

/*
 * ssa_index_topk without a workspace: the same indexer and top-k selection
 * (same arguments and results as ssa_index_topk, without scores_opt and ws),
 * for callers that cannot allocate device memory -- a plugin inside a host
 * program that owns every device allocation, or a serving loop that must not
 * allocate after start-up -- and so have no workspace to pass.
 *
 * The pages have no counterpart of this call; it only changes where the
 * score scratch lives.  That scratch is a fixed array of
 * SSA_STATIC_SCORE_ENTRIES int32 (4 MiB) compiled into the library, held on
 * every GPU that loads the library until the process exits.  A call needing
 * more than that (n_layers * batch * max_pages scores) returns
 * SSA_ERR_SCRATCH_LIMIT before enqueuing anything.  The call allocates and
 * frees nothing.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) and caches it: make that first call before
 * any stream capture.  Every call uses the same array, which keeps the last
 * call's scores; nothing in it needs clearing, but calls whose kernels
 * overlap on the GPU (other streams, other threads) race on it -- order them.
 */
#define SSA_STATIC_SCORE_ENTRIES (1u << 20)
int ssa_index_topk_static_scratch(const ssa_layout *lay, const ssa_cache *c, int layer0,
                                  int n_layers, const void *q, const int32_t *block_table,
                                  const int32_t *seq_lens, int32_t *sel, int32_t *n_sel,
                                  int32_t *status, ssa_stream_t stream);

/*
 * Failure-detection self-test (no counterpart in the pages): one CTA waits on
 * an mbarrier that nothing ever arrives on, using the bounded wait of every
 * kernel in this library (1 s of wall clock).  The wait gives up, the kernel
 * ORs SSA_ST_TIMEOUT into *status (device memory) and returns; the context
 * stays usable.  Takes about one second of GPU time.
 */
int ssa_selftest_bounded_wait(int32_t *status, ssa_stream_t stream);

/*
 * Measurement helper (no counterpart in the pages): the host link's rate for
 * reads issued by SMs, the access the miss fetch makes.  Copies n_chunks
 * chunks of chunk_bytes each, chunk i starting at byte offsets[i] of src,
 * into dst (chunk i at i * chunk_bytes), with 16-byte loads, loads_per_thread
 * (4, 8 or 16) in flight per thread, one group of 256-thread CTAs per chunk.
 *   src      pinned host memory the GPU can address (or device memory)
 *   dst      device memory, n_chunks * chunk_bytes bytes
 *   offsets  [n_chunks] int64, device memory; multiples of 16, and every
 *            chunk must lie inside the caller's source buffer (not checked:
 *            the values live on the device)
 * chunk_bytes a multiple of 16; 1 <= n_chunks <= 65535; src and dst 16-byte
 * aligned.  SSA_ERR_INVALID_ARG otherwise.  Time it with events on `stream`.
 */
int ssa_host_read_probe(const void *src, void *dst, const int64_t *offsets, int n_chunks,
                        int chunk_bytes, int loads_per_thread, ssa_stream_t stream);

/* Text for an SSA_ERR_* code or an SSA_ST_* bit set. */
const char *ssa_status_str(int code);

/* The cudaError_t of the last SSA_ERR_CUDA on this thread (0 if none). */
int ssa_last_cuda_error(void);

/* Number of kernel launches enqueued by calls on this thread so far. */
long long ssa_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* SSA_H */
