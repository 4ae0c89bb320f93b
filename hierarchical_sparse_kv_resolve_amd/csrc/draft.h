// The drafter's ring (kvr_draft) and its K/V layers in 8 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvr.h"

struct kvr_draft {
    int32_t n_req, W, C, R;
    uint8_t *ring;    // [n_req][C][R], or null: K/V layers only
    int32_t *length;  // [n_req]
    int32_t *high;    // [n_req]
    int device;
    // K/V layers (null codes: none bound)
    int32_t kv_layers, kv_heads, d_head;
    uint8_t *codes;   // [kv_layers][n_req][C / 64][kv_heads][2][64 * d_head]
    uint8_t *scales;  // [kv_layers][n_req][C / 64][kv_heads][2]
};

namespace kvr {

constexpr int kBlock = KVR_DRAFT_BLOCK;  // slots of a ring block
constexpr int kBias = 127;               // a scale byte b stands for 2^(b - kBias)
constexpr int kMinScale = kBias - 100;   // the smallest one

// One layer of a ring, as its kernels see it.
struct Window {
    int32_t n_req, W, C, blocks, kv_heads;  // blocks = C / 64
    uint8_t *codes;                         // the layer's
    uint8_t *scales;
    const int32_t *length, *high;
};

inline Window window_of(const kvr_draft *d, int32_t layer)
{
    Window w{};
    w.n_req = d->n_req;
    w.W = d->W;
    w.C = d->C;
    w.blocks = d->C / kBlock;
    w.kv_heads = d->kv_heads;
    const int64_t units = (int64_t)d->n_req * w.blocks * d->kv_heads * 2;
    w.codes = d->codes + layer * units * kBlock * d->d_head;
    w.scales = d->scales + layer * units;
    w.length = d->length;
    w.high = d->high;
    return w;
}

__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float(b << 23); }

// Entry i of a call: its request, lengths and number of new tokens, or why it
// is left out.
struct Entry {
    int32_t status, r, length, high, count;
};

__device__ __forceinline__ Entry entry_of(const Window &w, const int32_t *req_ids,
                                          const int32_t *count, int32_t rows, int i)
{
    Entry e{};
    e.r = req_ids ? req_ids[i] : i;
    e.count = count ? count[i] : rows;
    if (e.r < 0 || e.r >= w.n_req || e.count < 0 || e.count > rows) {
        e.status = KVR_E_ARG;
        return e;
    }
    e.length = w.length[e.r];
    e.high = w.high[e.r];
    if (e.length < 0 || e.high < e.length)
        e.status = KVR_E_STATE;
    else if (e.length > INT32_MAX - kBlock - e.count)  // (block ends stay in range)
        e.status = KVR_E_CAPACITY;
    return e;
}

int draft_prologue(const kvr_draft *d, int32_t n, hipStream_t s);

// Argument checks of the K/V calls: the ring and the stream's device; with them the layer.
int check_draft_stream(const kvr_draft *d, int32_t n, hipStream_t s);
int check_draft_kv(const kvr_draft *d, int32_t layer, int32_t n, hipStream_t s);

hipError_t launch_draft_write(const kvr_draft *d, const kvr_draft_write_call &c, hipStream_t s);
hipError_t launch_draft_read(const kvr_draft *d, int32_t layer, int32_t n, const int32_t *req_ids,
                             int32_t value_type, void *k, void *v, int32_t *visible,
                             int32_t *status, hipStream_t s);
hipError_t launch_draft_advance(const kvr_draft *d, int32_t n, const int32_t *req_ids,
                                int32_t rows, const int32_t *count, int32_t *status,
                                hipStream_t s);

// How a kvr_draft_attend call is cut: query rows (queries times the heads of one
// K/V head) per workgroup, whose waves share them (`split`: each wave takes other
// tokens) or have some each; shares of the tokens.
struct DraftPlan {
    int32_t blocks_of_16, waves, split, tiles, shares;
    int64_t workspace;
};
DraftPlan draft_plan(int32_t n, int32_t nq, int32_t heads, int32_t kv_heads, int32_t d_head,
                     int32_t tokens);
int64_t draft_workspace_bound(int32_t n, int32_t nq, int32_t heads, int32_t kv_heads,
                              int32_t d_head, int32_t window);
hipError_t launch_draft_attend(const kvr_draft *d, const kvr_draft_attend_call &c,
                               const DraftPlan &plan, hipStream_t s);

}  // namespace kvr
