/*
 * kvr.h - C ABI of the MI355X (gfx950) per-decode-step sparse KV row resolver.
 *
 * The method is the resolver of "Adaptive DHiSparse: Speculative Decoding over
 * a Load-Adaptive KV Hierarchy" (section "How it works"):
 *   - Memory split: each request has, per KV source, its own B-slot hot
 *     cache, a writable tail and its metadata; whole pages of the history it
 *     was admitted with may in addition be kept ready in an optional pool that
 *     all requests share.
 *   - Resolution: a selected row is taken from the first of three places that
 *     holds it: (1) the tail, else a ready page found through the optional
 *     page map; (2) the hot cache, whose lookup examines no more than B slots
 *     and which is managed LRU; (3) the pinned host store, from which the row
 *     is copied into a hot-cache slot.
 *   - Speculative state: the queries of one verification block fetch each
 *     missing row once between them.
 *   - Model-specific reuse: Reuse layers inherit a location vector when they
 *     share one physical KV source; layers that share sparse indices but own
 *     distinct payloads fetch the same positions for their own payload.
 *
 * One context serves one KV source: n_req requests and n_layers payload
 * layers that share the source's metadata (history length, page map, hot-cache
 * tags and stamps).
 *
 * Conventions
 *   - Every buffer is caller-owned.  Pointers marked (device) are device
 *     memory; (host) is ordinary host memory read during the call; (pinned) is
 *     page-locked host memory from hipHostMalloc (for example kvr_host_alloc or
 *     a pinned torch tensor), which kernels read and write directly over the
 *     host link.  The library keeps bound pointers until kvr_destroy and never
 *     frees them.
 *   - Calls that take a stream enqueue work on it (a hipStream_t; NULL is the
 *     default stream) and return without waiting for the device.  They never
 *     synchronise the host and allocate nothing.  Their return value reports
 *     argument errors only.
 *   - Data-dependent errors (a selected row outside [0, L), more distinct
 *     pending rows than B, a missing row without a host copy) are written per
 *     request into a device status array, stream-ordered.  A request that fails
 *     changes nothing: L, tags, stamps, clock and hot payload stay as they were
 *     and its locations read KVR_LOC_INVALID.  The other requests of the call
 *     complete normally.
 *   - Return codes are kvr_status values; kvr_last_error() gives a message for
 *     the calling thread's last failure.  No C++ exception leaves the library.
 *   - Threads and streams: the calls that launch work only read the context,
 *     so several host threads may issue them at once, except while launch
 *     timing is on (kvr_timing_begin to kvr_timing_end records into the
 *     context); kvr_bind_*, kvr_timing_* and kvr_destroy need the caller to
 *     keep every other call on that context out meanwhile.  On the device,
 *     calls that touch the same request must be ordered (one stream, or
 *     events between streams): two resolves of one request in flight at once
 *     race on its tags, stamps and clock.
 *
 * Location word (uint32): bits 31..30 give the place (kvr_place), bits 29..0
 * the index in it: the tail ring slot (pos mod T), the optional-pool row
 * (physical page * P + pos mod P) or the hot-cache slot.  A hot-cache word
 * carries KVR_LOC_FRESH (bit 29) when its row was copied from host memory by
 * the call that wrote the word; its slot is then in bits 28..0.
 */
#ifndef KVR_H
#define KVR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kvr_status {
    KVR_OK = 0,
    KVR_E_ARG = -1,          /* bad argument, shape or unbound buffer            */
    KVR_E_RANGE = -2,        /* selected row outside [0, L), or a bad location   */
    KVR_E_CAPACITY = -3,     /* more distinct pending rows than B; history full  */
    KVR_E_NO_HOST_COPY = -4, /* a missing row is neither on device nor on host   */
    KVR_E_HIP = -5,          /* the HIP runtime reported an error               */
    KVR_E_STATE = -6,        /* the LRU clock would wrap                         */
} kvr_status;

typedef enum kvr_place {
    KVR_PLACE_TAIL = 0,
    KVR_PLACE_PAGE = 1,
    KVR_PLACE_HOT = 2,
    KVR_PLACE_INVALID = 3,
} kvr_place;

#define KVR_LOC_INVALID 0xFFFFFFFFu
#define KVR_LOC_FRESH (1u << 29)  /* hot-cache word: filled from host by this call */

typedef enum kvr_reuse_mode {
    /* Reuse layers of one physical KV source: the location vector is inherited
     * as is (dst_loc NULL = alias, zero bytes moved; else a copy of it). */
    KVR_REUSE_SHARED_SOURCE = 0,
    /* Shared indices, distinct per-layer payloads: the rows filled from host
     * for one layer are fetched into the same hot slots of every destination
     * layer from that layer's host store; dst_loc (optional) receives a copy
     * of src_loc. */
    KVR_REUSE_DISTINCT_PAYLOAD = 1,
} kvr_reuse_mode;

/* Shape of one KV source.  Limits: 1 <= hot_slots <= 8192,
 * 1 <= sel_cap <= 8192, row_bytes a positive multiple of 16,
 * pool_pages * page_rows < 2^30, history_rows + max_new_rows < 2^31. */
typedef struct kvr_config {
    int32_t n_req;        /* requests of the source                           */
    int32_t n_layers;     /* payload layers sharing the source's metadata     */
    int32_t history_rows; /* H: imported history rows per request             */
    int32_t max_new_rows; /* decoded rows a request may append                */
    int32_t page_rows;    /* P: rows per optional-history page                */
    int32_t tail_rows;    /* T: rows in the mutable tail ring (0 = no tail)   */
    int32_t hot_slots;    /* B: hot-cache slots per request                   */
    int32_t row_bytes;    /* R: bytes per row (opaque payload)                */
    int32_t sel_cap;      /* most selection entries one request passes to one
                             resolve call (the union capacity for verify)     */
    int32_t reserved;     /* must be 0                                        */
    int64_t pool_pages;   /* pages in the global optional pool, per layer     */
} kvr_config;

/* One host refill: `row` was copied into hot slot `slot`. */
typedef struct kvr_fill {
    int32_t row;
    int32_t slot;
} kvr_fill;

/* Resolution counters, added to (device atomics) by every resolve call.
 * tail/page/hit/miss count selection entries by where they were found; fill
 * counts distinct rows copied from host and host_bytes their bytes. */
typedef struct kvr_stats {
    uint64_t calls, tail, page, hit, miss, fill, host_bytes, error;
} kvr_stats;

typedef struct kvr_ctx kvr_ctx;

/* Validate `cfg` and create a context on the current HIP device.  Allocates
 * only a small device table of layer pointers.  *out is NULL on failure. */
int kvr_create(const kvr_config *cfg, kvr_ctx **out);

/* Free the context (not the bound buffers).  NULL is accepted. */
int kvr_destroy(kvr_ctx *ctx);

/* Message for the calling thread's last non-OK return ("" if none). */
const char *kvr_last_error(void);

/* Bind the source's metadata (all device):
 *   L         int32  [n_req]              rows held: H + decoded rows
 *   page_map  int32  [n_req][ceil(H/P)]   physical page of a ready complete
 *                                          page, else -1 (a trailing partial
 *                                          page is never ready)
 *   host_valid uint8 [n_req][ceil(H/P)]   1 if the imported page has a host copy
 *   tag       int32  [n_req][B]           row held by a hot slot, -1 = empty
 *   stamp     uint32 [n_req][B]           LRU stamp of a hot slot
 *   clock     uint32 [n_req]              last LRU tick of the request
 * page_map and host_valid change only in kvr_reclaim_pages,
 * kvr_restore_pages and the calls on shared pages (kvr_release_requests,
 * kvr_fork_requests, kvr_copy_pages, kvr_compact_pool). */
int kvr_bind_metadata(kvr_ctx *ctx, int32_t *L, int32_t *page_map, uint8_t *host_valid,
                      int32_t *tag, uint32_t *stamp, uint32_t *clock);

/* Bind one payload layer:
 *   tail (device) [n_req][T][R], pool (device) [pool_pages][P][R] (written
 *   only by kvr_restore_pages, kvr_copy_pages and kvr_compact_pool),
 *   hot (device) [n_req][B][R], host (pinned) [n_req][H + max_new][R].
 * tail may be NULL when T = 0 and pool when pool_pages = 0. */
int kvr_bind_layer(kvr_ctx *ctx, int32_t layer, void *tail, void *pool, void *hot,
                   void *host);

/* Fresh admission: L = H, every tag -1, every stamp 0, every clock 0. */
int kvr_init_state(kvr_ctx *ctx, void *stream);

/* Append one decoded row to each listed request, for every layer: the row
 * goes to tail slot L mod T and, written through, to host row L; then L += 1.
 * Decoded rows never enter optional pages (section "Limits": they follow
 * hot-cache rules), which is why they get a host copy.
 *   req_ids  (device) int32 [n] or NULL (= 0..n-1); distinct
 *   new_rows (device) [n_layers][n][R]
 *   status   (device) int32 [n] or NULL: KVR_OK, or KVR_E_CAPACITY when the
 *            request already holds H + max_new rows (nothing written). */
int kvr_append_rows(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, const void *new_rows,
                    int32_t *status, void *stream);

/* Resolve one selection per listed request ("Resolution", steps 1-3).
 *   sel       (device) int32 [n][stride], rows of request i in sel[i][0..cnt)
 *   sel_count (device) int32 [n] or NULL (= stride); 0 <= cnt <= stride <= sel_cap
 *   loc       (device) uint32 [n][stride] out; entries >= cnt untouched
 *   fills     (device) kvr_fill [n][B] out: the rows copied from host, by
 *             ascending row; fill_count (device) int32 [n] out
 *   fill_layer payload layer refilled from host now, or -1 for none (the
 *             fills can be replayed into any layers with kvr_reuse_locations)
 *   status    (device) int32 [n] out, required
 *   stats     (device) kvr_stats or NULL, added to
 * Per request, with now = clock + 1 (one tick per call):
 *   1. a row in [max(0, L - T), L) is in the tail; else a row of a ready
 *      complete page is in the optional pool; else it is pending;
 *   2. each distinct pending row is looked for among the B tags; a hit
 *      stamps its slot with now;
 *   3. misses, by ascending row, take the slots not hit in this call with the
 *      smallest (stamp, slot), which get the row's tag and stamp now, and the
 *      host copy is fetched into them.
 * Repeated rows in one selection share one location. */
int kvr_resolve_rows(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, const int32_t *sel,
                     const int32_t *sel_count, int32_t stride, uint32_t *loc, kvr_fill *fills,
                     int32_t *fill_count, int32_t fill_layer, int32_t *status, kvr_stats *stats,
                     void *stream);

/* kvr_append_rows followed by kvr_resolve_rows for the same requests, in one
 * launch: each request's row is appended (tail slot L mod T, host row L,
 * L += 1) before its selection is resolved against the new length.  The
 * arguments are those of the two calls (new_rows and append_status as in
 * kvr_append_rows; append_status may be NULL).  An append that fails
 * (KVR_E_CAPACITY) changes nothing and the resolve still runs, as with the
 * two calls; an entry whose request id is out of range fails both; one whose
 * selection count is out of range fails its resolve (KVR_E_ARG) after its
 * append. */
int kvr_append_resolve_rows(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, const void *new_rows,
                            int32_t *append_status, const int32_t *sel, const int32_t *sel_count,
                            int32_t stride, uint32_t *loc, kvr_fill *fills, int32_t *fill_count,
                            int32_t fill_layer, int32_t *status, kvr_stats *stats, void *stream);

/* kvr_append_resolve_rows with the tail write of the append deferred, so
 * that the resolve of the next decode step may run while the previous step's
 * rows are still being gathered (the step's KV write, "Memory split": the
 * tail is the writable part; "Limits": decoded rows get a host copy).  The
 * launch writes each appended row's host copy and advances L, but leaves its
 * tail slot (L mod T) alone: that slot still holds the row L - T, which a
 * gather of the previous step may be reading.  append_pos (device) int32 [n]
 * receives, per entry, the position appended, or -1 when the entry appended
 * nothing (a failed append or a bad request id).  The resolve itself sees
 * the new length, exactly as after kvr_append_resolve_rows.  The appends are
 * completed by kvr_fused_gather_append_rows with the same entries, new_rows
 * and append_pos; until then a gather other than that one must not read the
 * tail slot of an appended row.  Other arguments and errors as for
 * kvr_append_resolve_rows. */
int kvr_append_resolve_rows_deferred(kvr_ctx *ctx, int32_t n, const int32_t *req_ids,
                                     const void *new_rows, int32_t *append_status,
                                     int32_t *append_pos, const int32_t *sel,
                                     const int32_t *sel_count, int32_t stride, uint32_t *loc,
                                     kvr_fill *fills, int32_t *fill_count, int32_t fill_layer,
                                     int32_t *status, kvr_stats *stats, void *stream);

/* Gather resolved rows into contiguous per-request buffers, for several
 * payload layers sharing one location vector ("Adaptive DHiSparse", section
 * "How it works", paragraph "Model-specific reuse": a layer reads its rows
 * where the location vector says; layers with shared sparse indices but
 * their own payloads each read their own bytes at the same locations):
 *   out[l] (device) [n][stride][R] for layers[l]; row j < cnt of request i is
 *   the R bytes at loc[i][j] in that layer (a fresh hot-cache row is read
 *   from its slot, so its fill must have run).  Invalid locations leave the
 *   row untouched.
 *   layers (host) int32 [n_layers]; out (host) array of n_layers device pointers
 *   loc (device) uint32 [n][stride]; count (device) int32 [n] or NULL (= stride)
 *   status (device) int32 [n] or NULL: set to KVR_E_RANGE for a request with a
 *   location outside its place, otherwise not written (clear it beforehand). */
int kvr_gather_rows(kvr_ctx *ctx, int32_t n_layers, const int32_t *layers, int32_t n,
                    const int32_t *req_ids, const uint32_t *loc, const int32_t *count,
                    int32_t stride, void *const *out, int32_t *status, void *stream);

/* The same gather split in two so that host fills and HBM gathers overlap
 * (same arguments as kvr_gather_rows; together the two write what
 * kvr_gather_rows writes after the fills):
 *   kvr_gather_resident_rows copies every row whose location is not a fresh
 *     hot-cache word (tail, page, hot-cache hit).  It reads no slot a fill of
 *     the same call writes, so it may run while those fills are in flight.
 *   kvr_fill_gather_rows copies every fresh row once from the layer's pinned
 *     host store into both the layer's hot-cache slot and the output: the
 *     host fill of that layer and its gather in one pass over the host link.
 *     sel (device) int32 [n][stride] is the selection the resolve call took
 *     (entry j's row); it reads no tag, so a later resolve of the same
 *     requests may run beside it.  Use it instead of fill_layer and
 *     kvr_reuse_locations(KVR_REUSE_DISTINCT_PAYLOAD) for these layers;
 *     repeated rows fetch their host copy once per repeat. */
int kvr_gather_resident_rows(kvr_ctx *ctx, int32_t n_layers, const int32_t *layers, int32_t n,
                             const int32_t *req_ids, const uint32_t *loc, const int32_t *count,
                             int32_t stride, void *const *out, int32_t *status, void *stream);
int kvr_fill_gather_rows(kvr_ctx *ctx, int32_t n_layers, const int32_t *layers, int32_t n,
                         const int32_t *req_ids, const uint32_t *loc, const int32_t *sel,
                         const int32_t *count, int32_t stride, void *const *out, int32_t *status,
                         void *stream);

/* kvr_fill_gather_rows and kvr_gather_resident_rows as one launch (same
 * arguments as kvr_fill_gather_rows; writes what the two write together):
 * part of the grid fills fresh rows from host while the rest gathers the
 * resident rows, with no wait between two launches on two streams.  Errors as
 * for the two calls. */
int kvr_fused_gather_rows(kvr_ctx *ctx, int32_t n_layers, const int32_t *layers, int32_t n,
                          const int32_t *req_ids, const uint32_t *loc, const int32_t *sel,
                          const int32_t *count, int32_t stride, void *const *out, int32_t *status,
                          void *stream);

/* kvr_fused_gather_rows that also completes the appends a
 * kvr_append_resolve_rows_deferred call left pending for the same entries
 * (same req_ids and n): for each entry with append_pos[i] >= 0, new_rows
 * (device) [n_layers of the context][n][R] row i of every layer goes into
 * tail slot append_pos[i] mod T, and a tail word of that entry naming that
 * slot is gathered from new_rows (the same bytes).  The call must name every
 * payload layer of the context exactly once (KVR_E_ARG otherwise), so every
 * layer's tail receives its row; with an empty selection (stride 0 or
 * counts 0) it still writes the rows.  Outputs and errors as for
 * kvr_fused_gather_rows. */
int kvr_fused_gather_append_rows(kvr_ctx *ctx, int32_t n_layers, const int32_t *layers, int32_t n,
                                 const int32_t *req_ids, const uint32_t *loc, const int32_t *sel,
                                 const int32_t *count, int32_t stride, void *const *out,
                                 int32_t *status, const void *new_rows, const int32_t *append_pos,
                                 void *stream);

/* One fused gather, as the arguments of kvr_fused_gather_append_rows
 * (new_rows and append_pos NULL: of kvr_fused_gather_rows).  layers and out
 * are host arrays of n_layers entries; the other pointers as documented
 * there. */
typedef struct kvr_gather_call {
    int32_t n_layers;
    const int32_t *layers;
    int32_t n;
    const int32_t *req_ids;
    const uint32_t *loc;
    const int32_t *sel;
    const int32_t *count;
    int32_t stride;
    void *const *out;
    int32_t *status;
    const void *new_rows;
    const int32_t *append_pos;
} kvr_gather_call;

/* One resolve, as the arguments of kvr_append_resolve_rows_deferred
 * (new_rows, append_status and append_pos NULL: of kvr_resolve_rows), with
 * no host fill (fill_layer -1). */
typedef struct kvr_resolve_call {
    int32_t n;
    const int32_t *req_ids;
    const void *new_rows;
    int32_t *append_status;
    int32_t *append_pos;
    const int32_t *sel;
    const int32_t *sel_count;
    int32_t stride;
    uint32_t *loc;
    kvr_fill *fills;
    int32_t *fill_count;
    int32_t *status;
    kvr_stats *stats;
} kvr_resolve_call;

/* The gather of one resolved selection and the resolve of the next one (the
 * next resolving layer's, or the next decode step's) in one launch ("How it
 * works": the resolve of "Resolution" and the gather the location vector of
 * "Model-specific reuse" feeds), so that the resolve leaves the critical
 * path without a wait between two queues.  Same results as
 * kvr_fused_gather_append_rows (or kvr_fused_gather_rows) with `gather`
 * followed by kvr_append_resolve_rows_deferred (or kvr_resolve_rows) with
 * `resolve`, provided the resolve writes none of the buffers the gather
 * reads (its loc, sel, count, new_rows and append_pos: give the two calls
 * different buffers, e.g. two sets used in turn).  The two never touch the
 * same state otherwise: the resolve reads and writes metadata and writes the
 * host copy of appended rows (beyond every row the gather fetches); the
 * gather writes hot-cache slots, tails and outputs.  An append in `resolve`
 * must be deferred (append_pos given): its tail slot may still be read by the
 * gather.  Either call may be NULL (then this is the other call alone);
 * argument errors of either half are returned before anything is launched.
 * Calls on one stream run in order, so a decode loop issues, per resolving
 * layer, this call with the previous layer's gather and this layer's
 * resolve, and ends with the last gather alone. */
int kvr_gather_resolve_rows(kvr_ctx *ctx, const kvr_gather_call *gather,
                            const kvr_resolve_call *resolve, void *stream);

/* Verification block dedup ("Speculative state": queries share missing-row
 * retrieval).  Per request: union_rows[i][0..u) = the distinct rows of the q
 * selections, ascending; map[i][qi][j] = index of sel[i][qi][j] in it.
 *   sel (device) int32 [n][q][k]; union_rows (device) int32 [n][q*k];
 *   union_count (device) int32 [n]; map (device) int32 [n][q][k].
 *   Requires q * k <= 8192.  The union is then resolved once. */
int kvr_dedup_verify_selections(kvr_ctx *ctx, int32_t n, int32_t q, int32_t k, const int32_t *sel,
                                int32_t *union_rows, int32_t *union_count, int32_t *map,
                                void *stream);

/* Location reuse across layers ("Model-specific reuse"); see kvr_reuse_mode.
 *   SHARED_SOURCE: dst_layers may be NULL; dst_loc (optional) gets src_loc.
 *   DISTINCT_PAYLOAD: the fills are replayed into every listed layer, all in
 *     one launch per 24 layers: row `row` of that layer's host store is copied
 *     into hot slot `slot` of that layer.
 *   dst_layers (host) int32 [n_layers]
 *   src_loc/dst_loc (device) uint32 [n][stride]; count (device) int32 [n] or NULL
 *   fills/fill_count (device): from the resolve call (DISTINCT_PAYLOAD only)
 *   status (device) int32 [n] or NULL: set to KVR_E_RANGE if a fill names a
 *   row or slot out of range, otherwise not written. */
int kvr_reuse_locations(kvr_ctx *ctx, int32_t mode, int32_t n_layers, const int32_t *dst_layers,
                        int32_t n, const int32_t *req_ids, const uint32_t *src_loc,
                        uint32_t *dst_loc, const int32_t *count, int32_t stride,
                        const kvr_fill *fills, const int32_t *fill_count, int32_t *status,
                        void *stream);

/* Optional-pool residency ("Adaptive DHiSparse", section "How it works",
 * paragraph "Reclamation and refill"): no row is ever lost, since a page
 * leaves the GPU only with a host backup in place and only once the kernels
 * that read it earlier are done; pages taken away are brought back later.
 *
 * kvr_reclaim_pages: the listed (req_ids[i], pages[i]) optional pages stop
 * being ready.  A page without a host copy first gets one (its P rows of
 * every payload layer are written from the pool to the host store over the
 * host link), then page_map becomes -1 and host_valid 1.  Stream order makes
 * the release wait for the kernels enqueued before it (earlier readers), and
 * every later kernel sees the page released.
 *   req_ids, pages (device) int32 [n]
 *   freed_phys (device) int32 [n]: the physical page entry i released, or -1
 *     if that page was not ready (also for a repeat of an earlier entry)
 *   status (device) int32 [n] or NULL: KVR_E_ARG for a request or page index
 *     out of range, KVR_E_STATE for a corrupt map entry (a physical page
 *     outside the pool, or an incomplete page marked ready; nothing moves),
 *     else KVR_OK.
 * kvr_restore_pages: the listed pages become ready in physical pages phys[i]:
 * their host rows of every layer are copied into the pool, then page_map
 * points at them.
 *   req_ids, pages, phys (device) int32 [n]; the caller hands out physical
 *     pages that no ready page maps (kvr_residency_refill does)
 *   status (device) int32 [n] or NULL: KVR_E_ARG for a request or page index
 *     out of range, a page that is not complete imported history, or a page
 *     or physical page that an earlier entry names; else KVR_E_RANGE for a
 *     physical page outside the pool; else KVR_E_STATE if the page is ready;
 *     else KVR_E_NO_HOST_COPY if it has no host copy; a failed entry changes
 *     nothing.
 * Both enqueue one kernel on `stream`; n = 0 is a no-op; n is at most
 * n_req * ceil(H/P). */
int kvr_reclaim_pages(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, const int32_t *pages,
                      int32_t *freed_phys, int32_t *status, void *stream);
int kvr_restore_pages(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, const int32_t *pages,
                      const int32_t *phys, int32_t *status, void *stream);

/* Formats of the rows a model's attention reads (every other call moves rows
 * as opaque bytes).  A row holds one token's latent (d_v values) and the
 * rotated part of its key (d_rope values); its key is both, its value the
 * latent, and every head shares it.
 *   KVR_ROW_BF16, KVR_ROW_F16: d_v + d_rope values of 16 bits
 *   KVR_ROW_FP8: d_v e4m3 codes, then one 32-bit scale for each 128 of them
 *     (the scales padded with zeros to a multiple of 16 bytes), then d_rope
 *     values of bf16.  A code stands for code * scale.
 * d_v is 256 or 512, d_rope 0 or 64. */
typedef enum kvr_row_format {
    KVR_ROW_BF16 = 0,
    KVR_ROW_F16 = 1,
    KVR_ROW_FP8 = 2,
} kvr_row_format;

/* Type of the values handed to kvr_pack_rows. */
typedef enum kvr_value_type {
    KVR_VALUE_BF16 = 0,
    KVR_VALUE_F16 = 1,
    KVR_VALUE_F32 = 2,
} kvr_value_type;

/* Bytes of one row of a format (1152 for 16-bit and 656 for fp8 rows of
 * d_v 512, d_rope 64), or KVR_E_ARG for a format or size not offered. */
int kvr_row_layout(int32_t format, int32_t d_v, int32_t d_rope);

/* Arguments of kvr_pack_rows.
 *   rows (device or pinned) [n][row_bytes] out, aligned to 16 bytes and
 *     disjoint from the inputs; row_bytes must be kvr_row_layout's
 *   latent (device) [n][d_v] of value_type, consecutive rows latent_stride
 *     elements apart; rope [n][d_rope] likewise (NULL when d_rope is 0);
 *     slices of one projection's output are taken as they are
 *   weight (device) float [d_v] or NULL: with it the latent is normalised,
 *     x = latent / sqrt(mean(latent^2) + eps) * weight (sums in 32 bits, so
 *     latents above about 8e17 overflow them and become 0); without it
 *     x = latent */
typedef struct kvr_pack_call {
    int32_t format;      /* kvr_row_format */
    int32_t value_type;  /* kvr_value_type */
    int32_t n;
    int32_t d_v;
    int32_t d_rope;
    float eps;
    const void *latent;
    const void *rope;
    const float *weight;
    void *rows;
    int64_t latent_stride;
    int64_t rope_stride;
} kvr_pack_call;

/* Rows of n new (or imported) tokens in the cache's format, for
 * kvr_append_rows, a host store or the optional pool.  x is rounded once, to
 * nearest, to the row's 16-bit type; in fp8 rows each group of 128 values has
 * scale = max|x| / 448 (1 for a group of zeros) and codes e4m3(x / scale)
 * (the quotient to 32-bit accuracy).  A scale below the smallest normal 32-bit
 * value is a whole number of 2^-149; quotients by one that is too small for
 * its group become the largest code, and one that rounds to 0 makes a group
 * of zeros.
 * The rope part is rounded to 16 bits as it is.  A NaN or an infinity makes
 * its own scale group (its own value, in 16-bit rows; the whole latent when
 * it is normalised) NaN or infinite, no other.  One kernel; n = 0 is a no-op. */
int kvr_pack_rows(kvr_ctx *ctx, const kvr_pack_call *call, void *stream);

/* Arguments of kvr_attend_rows.  Names shared with kvr_gather_rows mean the
 * same.
 *   rows, loc: where row j of request entry i is read.  rows (device)
 *     [n][stride][R] is a gathered buffer (kvr_gather_rows' out; aligned to 16
 *     bytes); with rows NULL the row is read where loc[i][j] names it in
 *     `layer` (tail, optional pool or hot cache, here aligned to 16 bytes; a
 *     fresh row's host fill must have run).  loc (device) uint32 [n][stride] is required with rows NULL;
 *     otherwise it may be NULL.  Entries whose word is KVR_LOC_INVALID are
 *     left out of the attention in both cases.
 *   count (device) int32 [n] or NULL (= stride): only entries j < count[i]
 *     are attended to
 *   map (device) int32 [n][nq][k] or NULL: with it (kvr_dedup_verify_selections'
 *     map) query a of entry i attends to the k entries map[i][a][0..k) of the
 *     union; indices outside [0, count[i]) are left out.  Without it (k is
 *     ignored) every query attends to all count[i] entries.
 *   q (device) [n][nq][heads][d_v + d_rope], 16-bit values of the format's type
 *     (bf16 with fp8 rows); strides in elements between entries, queries and
 *     heads, the last dimension contiguous
 *   out (device) [n][nq][heads][d_v] contiguous, of q's type, aligned to 16
 *     bytes, disjoint from the inputs; lse (device) float [n][nq][heads] or NULL
 *   status (device) int32 [n] or NULL: KVR_E_RANGE for an entry with a
 *     location outside its place (which is left out; rows NULL only),
 *     KVR_E_ARG for a request id out of range (which attends to nothing),
 *     otherwise not written
 *   workspace (device), aligned to 16 bytes: at least
 *     kvr_attend_workspace(n, nq, heads, d_v, rows per query) bytes; written
 *     by the call, so calls that may run at once (two streams, two graphs)
 *     each need their own */
typedef struct kvr_attend_call {
    int32_t layer;
    int32_t format;  /* kvr_row_format */
    int32_t n;
    int32_t nq;
    int32_t heads;
    int32_t d_v;
    int32_t d_rope;
    int32_t stride;
    int32_t k;
    float scale;
    const int32_t *req_ids;
    const uint32_t *loc;
    const void *rows;
    const int32_t *count;
    const int32_t *map;
    const void *q;
    int64_t q_stride_entry;
    int64_t q_stride_query;
    int64_t q_stride_head;
    void *out;
    float *lse;
    int32_t *status;
    void *workspace;
    size_t workspace_bytes;
} kvr_attend_call;

/* Attention of each request's new tokens over its resolved rows ("Adaptive
 * DHiSparse", section "How it works", paragraph "Model-specific reuse":
 * attention consumes the rows the location vector names):
 *   s_j = scale * (q . key_j),  out = sum_j exp(s_j - lse) value_j,
 *   lse = ln sum_j exp(s_j)
 * over the entries of the query (one that is named twice counts twice).  A
 * query without any, or whose scores are all -infinity, gets out = 0 and
 * lse = -infinity.  Rows left out are not read, whatever they hold; a NaN in
 * a row that takes part shows in the result.  Products of 16-bit values (an
 * e4m3 code is exact in bf16), sums, maxima and exponentials in 32 bits;
 * probabilities are rounded to 16 bits before their product with the values
 * (off by at most 2^-8 of each, with fp16 rows by 2^-11 of it or 2^-34 of the
 * largest).
 * A selection may be cut into shares that are attended to apart and joined in
 * a fixed order: results do not vary from run to run (another n, nq or heads
 * may cut it otherwise and round differently).  One kernel, or two with
 * shares.  Limits: nq and heads at most 4096, n * nq * heads at most 2^22,
 * stride and k at most 2^24. */
int kvr_attend_rows(kvr_ctx *ctx, const kvr_attend_call *call, void *stream);

/* Workspace bytes of kvr_attend_rows for calls of up to n entries, nq
 * queries, heads heads and `rows` rows per query (k with a map, stride without
 * one); 0 is possible.  Negative or too large arguments give KVR_E_ARG. */
int64_t kvr_attend_workspace(int32_t n, int32_t nq, int32_t heads, int32_t d_v, int32_t rows);

/* Rotary positions.  A head's rotated part is d_rot consecutive values, taken
 * as d_rot / 2 pairs (u, v); at position p pair i becomes
 *   u' = magnitude * (u cos a - v sin a),  v' = magnitude * (v cos a + u sin a),
 *   a = 2 pi p frequencies[i]
 * (inverse: a negated, which takes positions off again, and with them the
 * gradient of the outputs to that of the inputs).  p * frequency and its whole
 * turns are taken in 64 bits, the rest in 32; each value is rounded once, to
 * its type. */
typedef enum kvr_rope_layout {
    KVR_ROPE_INTERLEAVED = 0, /* pair i: values 2i and 2i + 1         */
    KVR_ROPE_HALF = 1,        /* pair i: values i and i + d_rot / 2   */
} kvr_rope_layout;

/* Heads of one tensor: x and out (device) [n][heads][d_head] of the call's
 * value type, strides in elements, the last dimension contiguous; values
 * [at, at + d_rot) of each head are rotated, the others copied.  out == x (with
 * x's strides) rotates in place and leaves the others alone; otherwise out is
 * disjoint from the inputs.  Strides of out with which its heads would overlap
 * are refused (x's may be 0).  heads 0: no such tensor. */
typedef struct kvr_rotate_part {
    const void *x;
    void *out;
    int64_t x_stride_token;
    int64_t x_stride_head;
    int64_t out_stride_token;
    int64_t out_stride_head;
    int32_t heads;
    int32_t d_head;
    int32_t at;
    int32_t reserved;  /* must be 0 */
} kvr_rotate_part;

/* Arguments of kvr_rotate_rows.
 *   positions (device) int32 [n]; frequencies (device) double [d_rot / 2], in
 *   turns per position (kvr_rope_frequencies); d_rot even, 2 to 1024
 *   query, key: the two tensors rotated at the same positions in one launch,
 *   such as the rope parts of a step's queries and of its new rows' key
 * Limits: n and each part's heads below 2^24, n * heads below 2^31. */
typedef struct kvr_rotate_call {
    int32_t value_type;  /* kvr_value_type */
    int32_t layout;      /* kvr_rope_layout */
    int32_t n;
    int32_t d_rot;
    float magnitude;
    int32_t inverse;
    const int32_t *positions;
    const double *frequencies;
    kvr_rotate_part query;
    kvr_rotate_part key;
} kvr_rotate_call;

/* Rotates queries and the rope parts of keys before kvr_attend_rows,
 * kvr_pack_rows, kvr_draft_write_kv or kvr_draft_attend take them.  One kernel;
 * n = 0 is a no-op. */
int kvr_rotate_rows(kvr_ctx *ctx, const kvr_rotate_call *call, void *stream);

/* Stretching of the frequencies for contexts longer than a model was trained
 * on, by `factor` >= 1:
 *   NONE    f_i = base^(-2i / d_rot) / (2 pi)
 *   LINEAR  f_i / factor (positions interpolated)
 *   BASE    base * factor^(d_rot / (d_rot - 2)) in place of base, which
 *           stretches the slowest pair by factor and the fastest not at all
 *   RAMP    f_i (1 - r_i) + f_i / factor * r_i, where r_i rises from 0 to 1
 *           over the pairs between those that turn beta_fast and beta_slow times
 *           in original_length positions: r_i = clamp((i - low) / (high - low)),
 *           pair(t) = d_rot ln(original_length / (2 pi t)) / (2 ln base),
 *           low = floor(pair(beta_fast)), high = ceil(pair(beta_slow)), both
 *           held to [0, d_rot - 1] and high at least low + 0.001; the magnitude is
 *           0.1 ln(factor) + 1 (1 in the other kinds) */
typedef enum kvr_rope_scaling {
    KVR_ROPE_NONE = 0,
    KVR_ROPE_LINEAR = 1,
    KVR_ROPE_BASE = 2,
    KVR_ROPE_RAMP = 3,
} kvr_rope_scaling;

/* Host helper: frequencies (host) double [d_rot / 2] and *magnitude (or NULL).
 * base > 1, factor >= 1; RAMP also takes original_length >= 1 and
 * beta_fast > beta_slow > 0, the other kinds ignore them. */
int kvr_rope_frequencies(int32_t d_rot, double base, int32_t scaling, double factor,
                         int32_t original_length, double beta_fast, double beta_slow,
                         double *frequencies, float *magnitude);

/* Arguments of kvr_token_logprobs.
 *   logits (device) [n][vocab] of value_type, rows logits_stride elements apart
 *   scale  multiplies the logits (1 / temperature); above 0, below 2^127
 *   tokens (device) int32 [n][m]: given tokens of each row, such as the one a
 *     drafter proposed; logprob (device) float [n][m] out
 *   lse, entropy (device) float [n] out, or NULL
 *   top_ids (device) int32 [n][top], top_logprob (device) float [n][top] out
 *   workspace (device), aligned to 16 bytes: at least
 *     kvr_logprob_workspace(n, vocab) bytes; written by the call, so calls that
 *     may run at once each need their own
 * Limits: n at most 2^20, vocab 1 to 2^24, m at most 2^16, top at most 64,
 * n * m below 2^31.  Outputs are contiguous and disjoint from the inputs. */
typedef struct kvr_logprob_call {
    int32_t value_type;  /* kvr_value_type */
    int32_t n;
    int32_t vocab;
    int32_t m;
    int32_t top;
    float scale;
    const void *logits;
    int64_t logits_stride;
    const int32_t *tokens;
    float *logprob;
    float *lse;
    float *entropy;
    int32_t *top_ids;
    float *top_logprob;
    void *workspace;
    size_t workspace_bytes;
} kvr_logprob_call;

/* Log probabilities of given tokens under each row of logits ("Adaptive
 * DHiSparse", section "How it works", paragraph "Speculative state": the
 * target model's rows of a verification block, or a drafter's), with x_j the
 * scaled logits:
 *   lse = ln sum_j exp(x_j),  logprob = x_token - lse,
 *   entropy = -sum_j p_j ln p_j,  p_j = exp(x_j - lse)
 * and the `top` tokens of the largest logits (as given, before the scale) with
 * their log probabilities, largest first, the lower token first among equals.
 * Logits of -infinity have probability 0 (log probability -infinity) and are
 * no alternatives; places past the last alternative get token -1 and
 * -infinity.  A token outside [0, vocab) has log probability -infinity.  A row of
 * -infinity alone has lse -infinity, entropy 0 and log probabilities
 * -infinity; one that holds a NaN or +infinity has NaN in every float and -1 in
 * every token.  32-bit sums in a fixed order: results do not vary from run to
 * run.  Two kernels; n = 0 is a no-op. */
int kvr_token_logprobs(kvr_ctx *ctx, const kvr_logprob_call *call, void *stream);

/* Workspace bytes of kvr_token_logprobs for calls of up to n rows of up to
 * vocab logits.  Bad sizes give KVR_E_ARG. */
int64_t kvr_logprob_workspace(int32_t n, int32_t vocab);

/* Pages shared between requests.
 *
 * A ready page is never written again, so several requests may map one
 * physical page.  refs (device) int32 [pool_pages] counts, for each physical
 * page, the page_map entries that name it; a page is free when its count is 0
 * (the calls treat a count below 0 as free too).
 *
 * kvr_bind_page_refs: bind the counts (NULL: none, as after kvr_create).
 *   While they are bound, kvr_reclaim_pages lowers the count of each page it
 *   releases (freed_phys[i] still names the page entry i let go of, which is
 *   free only once its count is 0) and kvr_restore_pages refuses a physical
 *   page whose count is not 0 with KVR_E_STATE and sets the count of each page
 *   it fills to 1.  kvr_residency_* keeps lists of its own, which do not
 *   follow the calls below, and expects each physical page in one map entry:
 *   give entries pages of their own (kvr_copy_pages) before a map is handed to
 *   it.
 * kvr_count_page_refs: set the counts from page_map.
 *
 * The calls below need the counts bound when pool_pages > 0.
 *
 * kvr_release_requests: each listed request gives up its rows: the counts of
 *   its pages go down, page_map becomes -1, host_valid 0, tags -1, stamps 0,
 *   clock 0 and L 0, so that every row of it is out of range until it becomes
 *   the copy of another request or is set up again.  Payload stays as it is.
 *   What was resolved for a request before (its host fills, gathers, deferred
 *   appends) must have run before it is set up again or forked into.
 *   status (device) int32 [n] or NULL: KVR_E_ARG (nothing changes) for an id
 *   out of range or one that an earlier entry names.
 * kvr_fork_requests: request dst_ids[i] becomes a copy of src_ids[i]: L,
 *   clock, tags and stamps; the ready pages, shared; and of every payload layer
 *   the tail ring, the hot slots with a tag, the host rows of imported pages
 *   that have a host copy and are not ready, and those of decoded rows.  What
 *   dst held before is given up as by kvr_release_requests.  In the copy a
 *   ready page has no host copy (its backup is made when it is reclaimed).
 *   The host fills of the source's last resolve may still be outstanding (the
 *   slots it used are copied from their rows' host copies); fills of earlier
 *   resolves and deferred appends of the source must have been completed.  A
 *   drafter's window (kvr_draft_*) is a state of its own and not copied.
 *   src_ids, dst_ids (device) int32 [n]; a request may be the source of several
 *   entries.  status (device) int32 [n] or NULL: KVR_E_ARG (nothing changes)
 *   for an id out of range, a destination that an earlier entry names or a
 *   request that is both a source and a destination of the call.
 * kvr_copy_pages: request req_ids[i]'s ready page pages[i] is copied into
 *   physical page phys[i], which it maps from then on; the old page's count
 *   goes down.  status (device) int32 [n], required: KVR_E_ARG for a request or
 *   page out of range, an incomplete page, or a page or physical page that an
 *   earlier entry names; else KVR_E_RANGE for a physical page outside the pool;
 *   else KVR_E_STATE for a page that is not ready or a physical page in use.
 *   Entries are judged on the state before the call; a failed one changes
 *   nothing.
 * kvr_list_free_pages: free_list (device) int32 [pool_pages] receives the free
 *   physical pages, ascending, in its first free_count[0] (device) entries;
 *   the others are not written.
 * kvr_compact_pool: while free pages lie below live ones, the highest live
 *   page moves into the lowest free one, at most max_moves times: the payload
 *   of every layer, its count and every page_map entry naming it.  moves
 *   (device) int32 [min(max_moves, pool_pages)][2] receives (source,
 *   destination) of each in that order, move_count (device) int32 [1] their
 *   number.  After a call that reached no limit the live pages are the lowest.
 *   Location words resolved before it that name pages no longer hold: no
 *   compaction between a resolve and the gathers and attention that use it.
 *   workspace (device), aligned to 4 bytes: kvr_pool_workspace(ctx) bytes, for
 *   calls that may run at once one each.
 * n is at most n_req for lists of requests, min(n_req * ceil(H/P), 65536) for
 * lists of pages; n = 0 is a no-op. */
int kvr_bind_page_refs(kvr_ctx *ctx, int32_t *refs);
int kvr_count_page_refs(kvr_ctx *ctx, void *stream);
int kvr_release_requests(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, int32_t *status,
                         void *stream);
int kvr_fork_requests(kvr_ctx *ctx, int32_t n, const int32_t *src_ids, const int32_t *dst_ids,
                      int32_t *status, void *stream);
int kvr_copy_pages(kvr_ctx *ctx, int32_t n, const int32_t *req_ids, const int32_t *pages,
                   const int32_t *phys, int32_t *status, void *stream);
int64_t kvr_pool_workspace(const kvr_ctx *ctx);
int kvr_list_free_pages(kvr_ctx *ctx, int32_t *free_list, int32_t *free_count, void *workspace,
                        size_t workspace_bytes, void *stream);
int kvr_compact_pool(kvr_ctx *ctx, int32_t max_moves, int32_t *moves, int32_t *move_count,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Host-side residency policy of one KV source's optional pool (no device
 * work; the caller applies its decisions with the two calls above).
 *
 * kvr_residency_create: page_map (host) int32 [n_req][n_pages] the initial
 *   map, of which the first n_complete pages per request may be optional;
 *   pool_pages physical pages in the pool, those no page maps are free.
 * kvr_residency_admit: an admission needing `need` physical pages.  Free
 *   pages are used first; the pages still missing (the shortfall) come from
 *   requests that give up every ready page they hold, one request at a time
 *   in `order` (n_order request ids, the reclaim order), until enough are
 *   free; the requests after that keep theirs.  The lowest free page ids are
 *   reserved for the admission.  Writes the (request, page) list to reclaim,
 *   in that order (at most `cap` entries), and a handle.  Returns
 *   KVR_E_CAPACITY when the shortfall is larger than all optional pages
 *   together (the admission waits; nothing changes, *n_out = 0),
 *   KVR_E_ARG when the list would exceed `cap` (nothing changes).
 * kvr_residency_release: the admission drained; its pages are free again.
 * kvr_residency_refill: bounded round-robin refill of the pages that
 *   reclamation took (residency repopulates as load drains): requests are
 *   visited cyclically from a cursor kept between calls, each visit giving
 *   one request its lowest-index reclaimed page not yet back and the lowest
 *   free physical page, until `bound` pages (at most `cap`), no free page, or
 *   a whole cycle without such a page; the cursor then points after the last
 *   request served.  Pages not ready at creation are never refilled.  Writes
 *   (request, page, physical page) triples.
 * kvr_residency_counts: free, ready and reserved physical pages.
 * The object is not thread-safe. */
typedef struct kvr_residency kvr_residency;

int kvr_residency_create(int32_t n_req, int32_t n_pages, int32_t n_complete, int64_t pool_pages,
                         const int32_t *page_map, kvr_residency **out);
int kvr_residency_destroy(kvr_residency *res);
int kvr_residency_admit(kvr_residency *res, int64_t need, int32_t n_order, const int32_t *order,
                        int32_t cap, int32_t *req_out, int32_t *page_out, int32_t *n_out,
                        int32_t *handle);
int kvr_residency_release(kvr_residency *res, int32_t handle);
int kvr_residency_refill(kvr_residency *res, int32_t bound, int32_t cap, int32_t *req_out,
                         int32_t *page_out, int32_t *phys_out, int32_t *n_out);
int kvr_residency_counts(const kvr_residency *res, int64_t *free_pages, int64_t *ready_pages,
                         int64_t *reserved_pages);

/* Speculative state ("Adaptive DHiSparse", section "How it works",
 * paragraph "Speculative state").
 *
 * Drafter visible-window ring: the drafter stores no more than the rows it can
 * still see.  Per
 * request, drafter rows are numbered by position; row p lives in slot p mod C
 * of a ring of C >= W slots; the visible window is the last min(W, length)
 * positions.  The C - W extra slots let rows that verification rejects be
 * dropped: a rollback to a shorter length is allowed while no position
 * written since (kept or dropped) has overwritten the window it leaves
 * visible, i.e. for keep >= (highest position ever written + 1) - (C - W).
 *   kvr_draft_create: ring (device) [n_req][C][row_bytes] (row_bytes a
 *     multiple of 16), length and high (device) int32 [n_req] (rows kept, and
 *     highest position ever written + 1); all caller-owned; the current device
 *     is the ring's.  A drafter that keeps its rows in K/V layers only
 *     (kvr_draft_bind_kv) passes a NULL ring and row_bytes 0; append and window
 *     are refused then.  kvr_draft_reset zeroes length and high (stream-ordered).
 *   kvr_draft_append: rows (device) [n][rows_each][row_bytes], rows_each <= C,
 *     appended at positions length .. length + rows_each - 1.
 *   kvr_draft_rollback: keep (device) int32 [n]; status KVR_E_RANGE (nothing
 *     changes) when keep is above the length or below the rollback limit.
 *   kvr_draft_window: out (device) [n][W][row_bytes] receives the visible rows
 *     oldest first (rows past the window are untouched); visible (device)
 *     int32 [n] or NULL receives their number.
 *   status (device) int32 [n] or NULL: KVR_E_ARG for a request out of range.
 * req_ids (device) int32 [n] or NULL (= 0 .. n-1) name each request at most
 * once per call.  All calls enqueue one kernel on `stream` and never
 * synchronise the host. */
typedef struct kvr_draft kvr_draft;

int kvr_draft_create(int32_t n_req, int32_t window, int32_t capacity, int32_t row_bytes,
                     void *ring, int32_t *length, int32_t *high, kvr_draft **out);
int kvr_draft_destroy(kvr_draft *d);
int kvr_draft_reset(kvr_draft *d, void *stream);
int kvr_draft_append(kvr_draft *d, int32_t n, const int32_t *req_ids, int32_t rows_each,
                     const void *rows, int32_t *status, void *stream);
int kvr_draft_rollback(kvr_draft *d, int32_t n, const int32_t *req_ids, const int32_t *keep,
                       int32_t *status, void *stream);
int kvr_draft_window(kvr_draft *d, int32_t n, const int32_t *req_ids, void *out,
                     int32_t *visible, int32_t *status, void *stream);

/* The drafter's keys and values in 8 bits, in the same ring: position p lies in
 * slot p mod C of every layer, and length, high, window and rollback are the
 * ring's.  A ring block is KVR_DRAFT_BLOCK (64) slots; in each layer it holds,
 * for each K/V head, the keys [64][d_head] and the values [d_head][64] (a
 * dimension's 64 tokens side by side) as e4m3 codes, and one scale for the keys
 * and one for the values, a byte b that stands for 2^(b - 127).
 *   kvr_draft_bind_kv: codes (device, aligned to 16 bytes)
 *     [n_layers][n_req][C / 64][kv_heads][2][64 * d_head], scales (device) uint8
 *     [n_layers][n_req][C / 64][kv_heads][2]; C must be a multiple of 64,
 *     kv_heads 1 to 256, d_head 64, 128 or 256.  Needs every other call on this
 *     ring out meanwhile.
 *   kvr_draft_write_kv: new tokens of one layer at positions length ..
 *     length + count - 1, for kvr_draft_attend to see; length stays, so that
 *     every layer of a step writes at the same positions, until
 *     kvr_draft_advance.  A block's scale becomes the smallest power of two
 *     (2^-100 at least) with which its largest value is at most 448, over
 *     the rows it then holds: new ones and those kept.  New values are
 *     rounded once, to the nearest code (magnitudes that would become 2^128, from
 *     248 * 2^120 on, to 240 * 2^120, so that rows read back are finite in 32 bits
 *     and in bf16); codes of rows kept are moved to a
 *     changed scale, which is exact but for values that fall below the smallest
 *     normal code.  Slots of a touched block that hold no row (not written yet,
 *     or dropped by a rollback) become 0, others are left as they were.  A token
 *     whose key or value in a head holds a NaN or an infinity gets a key of NaN
 *     codes there and zeros for such values: it shows as NaN in the queries that
 *     see it, and in no others.
 *   kvr_draft_read_kv: the visible rows of one layer, oldest first, as
 *     kvr_draft_window; code * scale in the type asked for (exact in 32 bits
 *     and in bf16).  Status KVR_E_RANGE for an entry of which a visible row has
 *     been overwritten by a later one.  The ring learns of written tokens by
 *     kvr_draft_advance: before it, where more than C - W are written, the oldest
 *     rows seen by this call, and by queries of KVR_DRAFT_KEPT, are already those
 *     tokens, with status KVR_OK.
 *   kvr_draft_advance: length += count and high follows, once the layers have
 *     written their tokens (kvr_draft_append does the same, for a drafter with
 *     rows of both kinds: its K/V layers are written first).  What is drafted and
 *     rejected is dropped with kvr_draft_rollback: written tokens overwrite the
 *     rows C positions before them, which high has to know of, so they are
 *     advanced over before others are written in their place.
 * count (device) int32 [n] or NULL (= rows): new tokens of entry i, 0 to rows;
 * the inputs and outputs of the others are neither read nor written.
 * status (device) int32 [n] or NULL: KVR_OK; KVR_E_ARG for a request or a count
 * out of range; KVR_E_STATE for a length below 0 or above high; KVR_E_CAPACITY
 * for a length that would pass 2^31 - 65; such entries change and write nothing
 * else. */
#define KVR_DRAFT_BLOCK 64

int kvr_draft_bind_kv(kvr_draft *d, int32_t n_layers, int32_t kv_heads, int32_t d_head,
                      void *codes, uint8_t *scales);

/* Arguments of kvr_draft_write_kv: k, v (device) [n][rows][kv_heads][d_head] of
 * value_type, strides in elements between entries, tokens and heads, the last
 * dimension contiguous (slices of one projection's output are taken as they
 * are).  rows at most C - 63, so that no block is touched twice. */
typedef struct kvr_draft_write_call {
    int32_t layer;
    int32_t value_type;  /* kvr_value_type */
    int32_t n;
    int32_t rows;
    const int32_t *req_ids;
    const int32_t *count;
    const void *k;
    const void *v;
    int64_t k_stride_entry;
    int64_t k_stride_token;
    int64_t k_stride_head;
    int64_t v_stride_entry;
    int64_t v_stride_token;
    int64_t v_stride_head;
    int32_t *status;
} kvr_draft_write_call;

int kvr_draft_write_kv(kvr_draft *d, const kvr_draft_write_call *call, void *stream);

/* k, v (device) [n][W][kv_heads][d_head] of value_type, contiguous, aligned to
 * 16 bytes; visible (device) int32 [n] or NULL receives the number of rows. */
int kvr_draft_read_kv(kvr_draft *d, int32_t layer, int32_t n, const int32_t *req_ids,
                      int32_t value_type, void *k, void *v, int32_t *visible, int32_t *status,
                      void *stream);

int kvr_draft_advance(kvr_draft *d, int32_t n, const int32_t *req_ids, int32_t rows,
                      const int32_t *count, int32_t *status, void *stream);

/* Which rows query j of an entry sees: the last W (or fewer) rows before
 * position `end`. */
typedef enum kvr_draft_mask {
    KVR_DRAFT_CAUSAL = 0, /* end = length + j + 1: the tokens up to its own   */
    KVR_DRAFT_WHOLE = 1,  /* end = length + count: all of the new tokens      */
    KVR_DRAFT_KEPT = 2,   /* end = length: none of them (they need no row)   */
} kvr_draft_mask;

/* Arguments of kvr_draft_attend.
 *   q (device) bf16 [n][nq][heads][d_head], strides in elements, the last
 *     dimension contiguous; query head h reads K/V head h / (heads / kv_heads)
 *   count (device) int32 [n] or NULL (= nq): queries of entry i (and new tokens
 *     that kvr_draft_write_kv wrote); those past it are not read, their outputs
 *     not written
 *   out (device) bf16 [n][nq][heads][d_head] contiguous, aligned to 16 bytes,
 *     disjoint from the inputs; lse (device) float [n][nq][heads] or NULL
 *   status as above, and KVR_E_RANGE for an entry of which a query sees a row
 *     that a later one has overwritten (after a rollback)
 *   workspace (device), aligned to 16 bytes: at least
 *     kvr_draft_attend_workspace(d, n, nq, heads) bytes; written by the call, so
 *     calls that may run at once each need their own
 * heads is a multiple of kv_heads, at most 4096; n * nq * heads at most 2^22;
 * |scale| below 2^127; with KVR_DRAFT_CAUSAL nq is at most C - W + 1, with
 * KVR_DRAFT_WHOLE at most C. */
typedef struct kvr_draft_attend_call {
    int32_t layer;
    int32_t mask;  /* kvr_draft_mask */
    int32_t n;
    int32_t nq;
    int32_t heads;
    float scale;
    const int32_t *req_ids;
    const int32_t *count;
    const void *q;
    int64_t q_stride_entry;
    int64_t q_stride_query;
    int64_t q_stride_head;
    void *out;
    float *lse;
    int32_t *status;
    void *workspace;
    size_t workspace_bytes;
} kvr_draft_attend_call;

/* Attention of new tokens' queries over the drafter's window:
 *   s_j = scale * (q . key_j),  out = sum_j exp(s_j - lse) value_j,
 *   lse = ln sum_j exp(s_j)
 * over the rows the query sees; one that sees none gets out = 0 and
 * lse = -infinity.  Codes are exact in bf16; products, sums, maxima and
 * exponentials in 32 bits; probabilities are rounded to bf16 before their product
 * with the values.  Sums are divided at the end and weigh a row by 2^8 at most: they
 * are sure not to overflow while the values are below 2^120 / W.  Rows may be cut
 * into shares that are joined in a fixed order: results do not vary from run to run
 * (another n, nq or heads may cut them otherwise).  One kernel, or two with shares;
 * n = 0 is a no-op. */
int kvr_draft_attend(kvr_draft *d, const kvr_draft_attend_call *call, void *stream);

/* Workspace bytes of kvr_draft_attend calls of up to n entries, nq queries and
 * heads heads on this ring; 0 is possible.  Bad sizes give KVR_E_ARG. */
int64_t kvr_draft_attend_workspace(const kvr_draft *d, int32_t n, int32_t nq, int32_t heads);

/* Verification staging reuse: a target layer's staging buffer is handed out
 * again only after the kernels that read it have finished.  A pool of n_buffers caller-owned buffers, named by
 * index and handed out round-robin.  kvr_staging_acquire makes `stream` wait
 * until the buffer's previous consumer has released it; kvr_staging_release
 * records that release on the consumer's stream after its last read of the
 * buffer.  Host object, not thread-safe; acquire and release enqueue only an
 * event wait or record.  Not meant for graph capture (a release recorded
 * before the capture is not visible to it). */
typedef struct kvr_staging kvr_staging;

int kvr_staging_create(int32_t n_buffers, kvr_staging **out);
int kvr_staging_destroy(kvr_staging *p);
int kvr_staging_acquire(kvr_staging *p, void *stream, int32_t *index);
int kvr_staging_release(kvr_staging *p, int32_t index, void *stream);

/* Host helper, after the caller has synchronised and copied status to host:
 * number of failed requests; *first_bad = index of the first (or -1). */
int kvr_status_summary(const int32_t *status, int32_t n, int32_t *first_bad);

/* Page-locked, device-mapped host memory for host stores (hipHostMalloc).
 * Returns KVR_E_HIP on failure. */
int kvr_host_alloc(size_t bytes, void **out);
int kvr_host_free(void *ptr);

/* Kernel launch timing (measurement aid, not part of the method).
 *
 * Between kvr_timing_begin and kvr_timing_end every kernel the context
 * launches carries a start and a stop event of its own dispatch
 * (hipExtLaunchKernel), so each recorded duration is the kernel's execution
 * alone, the interval a kernel-trace profiler reports, without the gaps
 * between launches.  Launches on a stream that is being captured into a graph
 * are not recorded.
 *
 * kvr_timing_begin: capacity = most launches to record (1 .. 1048576).
 *   Creates the events when the context has fewer than that (this is the
 *   only call here that allocates), then starts recording; launches past the
 *   capacity run untimed and are counted.
 * kvr_timing_end: stops recording, waits for the recorded launches and
 *   writes, for each in launch order, kinds[i] (kvr_kernel) and ms[i] (host
 *   arrays of `capacity` entries); *n_recorded = launches recorded.  Returns
 *   KVR_E_CAPACITY if launches went untimed or did not fit the arrays (the
 *   entries that fit are still written), KVR_E_ARG if recording was not on. */
typedef enum kvr_kernel {
    KVR_KERNEL_APPEND = 0,
    KVR_KERNEL_RESOLVE = 1,
    KVR_KERNEL_REFILL = 2,   /* host refill and per-layer replays */
    KVR_KERNEL_GATHER = 3,
    KVR_KERNEL_DEDUP = 4,
    KVR_KERNEL_STATE = 5,    /* state initialisation, location copies */
    KVR_KERNEL_FUSED = 6,    /* fill pass and resident gather in one launch */
    KVR_KERNEL_STEP = 7,     /* a fused gather beside the next resolve */
    KVR_KERNEL_ATTEND = 8,   /* attention over resolved rows, and the join of its shares */
    KVR_KERNEL_PACK = 9,     /* rows of new tokens */
    KVR_KERNEL_PAGES = 10,   /* fork, release, page copies, free list, compaction */
    KVR_KERNEL_ROTATE = 11,  /* rotary positions */
    KVR_KERNEL_LOGPROB = 12, /* log probabilities, and the join of their parts */
} kvr_kernel;

int kvr_timing_begin(kvr_ctx *ctx, int32_t capacity);
int kvr_timing_end(kvr_ctx *ctx, int32_t capacity, int32_t *kinds, float *ms,
                   int32_t *n_recorded);

#ifdef __cplusplus
}
#endif

#endif /* KVR_H */
