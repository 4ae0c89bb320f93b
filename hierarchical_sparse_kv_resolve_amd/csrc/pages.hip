// Pages shared between requests: forking a request, freeing one, giving an
// entry a page of its own, and compacting the optional pool ("Adaptive
// DHiSparse: Speculative Decoding over a Load-Adaptive KV Hierarchy", section
// "How it works", paragraph "Memory split": complete pages of imported
// history live in one pool that all requests share).
//
// A ready page is complete imported history and is never written again, so
// any number of requests may map one physical page: a fork shares its
// source's ready pages and copies only what is the request's own (tail ring,
// filled hot slots, and the host rows no ready page covers).  refs[ph] counts
// the map entries naming physical page ph; a page is free when it is 0.  All
// counts change by integer atomics, so results do not depend on their order.
//
// Every kernel here moves whole rows or pages as 16-byte chunks and is bound
// by the memory it moves.  Measured on one MI355X:
//   fork      one request of 4096 rows of 1152 bytes, half of its pages ready
//             (2.4 MB read from and written to host memory, 1.2 MB of HBM
//             copies): 88 us; four requests of 8192 rows, two layers (22 MB each
//             way over the host link): 562 us, 80 GB/s of both directions (a
//             copy engine reaches 57 each way, two at once 57 together), 594
//             where the last resolve used half of the hot slots, whose rows are
//             then read from the host.  A tile of rows per workgroup; workers
//             in a loop (16 to 256) and 2 to 8 chunks a lane were no faster.
//   compact   256 pages of 73 KB, 30 % free: 8 us to rank them, 5 to move about
//             50 (an empty kernel 4); 16384 pages of 42 KB, about 3440 of them
//             moved (289 MB): 6 + 10 us to count and rank, 60 to move, 4.8 TB/s
//   copies    32 pages of 73 KB, two layers: 9 + 5 us in a trace of single
//             calls, 7 + 4 by events among calls issued back to back
//   counts    64 requests' maps over 16384 pages: 1.8 + 2.7 us
#include "kvr_internal.h"
#include "rows.h"

namespace kvr {
namespace {

constexpr int NT = kRowThreads;
constexpr int kFullGrid = 1024;          // workgroups that keep the card busy
constexpr int kMaxCopyBlocks = 1 << 16;  // grids past this stride over their jobs

// Whether an earlier entry of either list names id (every thread scans a
// share; the result is uniform).
__device__ bool named_earlier(const int32_t *ids, int i, int32_t id)
{
    bool hit = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x)
        hit |= ids[j] == id;
    return __syncthreads_or(hit);
}

__device__ bool named_anywhere(const int32_t *ids, int n, int32_t id)
{
    return named_earlier(ids, n, id);
}

__device__ __forceinline__ bool in_pool(const Shape &sh, int32_t ph)
{
    return ph >= 0 && (int64_t)ph * sh.P < sh.pool_rows;
}

// ---------------------------------------------------------------- counting

__global__ __launch_bounds__(NT) void zero_kernel(int32_t *p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < n; i += (int64_t)gridDim.x * NT)
        p[i] = 0;
}

__global__ __launch_bounds__(NT) void count_refs_kernel(Shape sh, const int32_t *page_map,
                                                        int32_t *refs)
{
    const int64_t n = (int64_t)sh.n_req * sh.n_pages;
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < n; i += (int64_t)gridDim.x * NT) {
        const int32_t ph = page_map[i];
        if (in_pool(sh, ph))
            atomicAdd(&refs[ph], 1);
    }
}

// ----------------------------------------------------------- release, fork

struct MetaPtrs {
    int32_t *L, *page_map;
    uint8_t *host_valid;
    int32_t *tag;
    uint32_t *stamp, *clock;
    int32_t *refs;
};

// One workgroup per listed request: its pages' counts go down and its state
// becomes that of a request without rows.
__global__ __launch_bounds__(NT) void release_kernel(Shape sh, MetaPtrs m, const int32_t *ids,
                                                     int32_t *status)
{
    const int i = blockIdx.x;
    const int32_t r = ids[i];
    const bool bad = r < 0 || r >= sh.n_req || named_earlier(ids, i, r);
    if (!bad) {
        for (int p = threadIdx.x; p < sh.n_pages; p += NT) {
            const int64_t e = (int64_t)r * sh.n_pages + p;
            const int32_t ph = m.page_map[e];
            if (in_pool(sh, ph))
                atomicSub(&m.refs[ph], 1);
            m.page_map[e] = -1;
            m.host_valid[e] = 0;
        }
        for (int b = threadIdx.x; b < sh.B; b += NT) {
            m.tag[(int64_t)r * sh.B + b] = -1;
            m.stamp[(int64_t)r * sh.B + b] = 0;
        }
    }
    if (threadIdx.x == 0) {
        if (!bad) {
            m.L[r] = 0;
            m.clock[r] = 0;
        }
        if (status)
            status[i] = bad ? KVR_E_ARG : KVR_OK;
    }
}

struct ForkArgs {
    Shape sh;
    MetaPtrs m;
    TileShape ts;
    const LayerPtrs *layers;  // device table
    const int32_t *src, *dst;
    int32_t *status;
    int32_t n;
    int32_t host_tiles, hot_tiles, tail_tiles;  // row tiles per (pair, layer)
};

// The metadata of one pair.  Ready pages are shared; a page the source keeps
// both ready and on the host is ready only in the copy, whose host backup is
// then made when the page is reclaimed.
__device__ void fork_metadata(const ForkArgs &a, int i, int32_t s, int32_t d)
{
    const Shape &sh = a.sh;
    for (int p = threadIdx.x; p < sh.n_pages; p += NT) {
        const int64_t es = (int64_t)s * sh.n_pages + p, ed = (int64_t)d * sh.n_pages + p;
        const int32_t was = a.m.page_map[ed], ph = a.m.page_map[es];
        if (in_pool(sh, was))
            atomicSub(&a.m.refs[was], 1);
        if (in_pool(sh, ph))
            atomicAdd(&a.m.refs[ph], 1);
        a.m.page_map[ed] = ph;
        a.m.host_valid[ed] = ph < 0 ? a.m.host_valid[es] : 0;
    }
    for (int b = threadIdx.x; b < sh.B; b += NT) {
        a.m.tag[(int64_t)d * sh.B + b] = a.m.tag[(int64_t)s * sh.B + b];
        a.m.stamp[(int64_t)d * sh.B + b] = a.m.stamp[(int64_t)s * sh.B + b];
    }
    if (threadIdx.x == 0) {
        a.m.L[d] = a.m.L[s];
        a.m.clock[d] = a.m.clock[s];
        if (a.status)
            a.status[i] = KVR_OK;
    }
}

// Whether row pos of request s has a host copy.
__device__ __forceinline__ bool host_copy(const ForkArgs &a, int32_t s, int32_t pos)
{
    const Shape &sh = a.sh;
    return pos < a.m.L[s] && pos < sh.host_rows &&
           (pos >= sh.H || a.m.host_valid[(int64_t)s * sh.n_pages + pos / sh.P]);
}

// A slot's tag is written by the resolve, its bytes by the fills that follow
// it, in each layer at its own time.  So slots that the source's last resolve
// used (their stamp is its clock) are read from their rows' host copies, which
// is what its fills bring.  (Without a host copy such a slot is not waiting for
// a fill: it is itself a copy, in a request forked since that resolve.)
//
// Jobs: per pair one of metadata, then row tiles of every layer: host rows
// first (the host link is the slow side), then hot slots and the tail.  No
// source is a destination of the same call, so what a job reads is not
// written by another.
__global__ __launch_bounds__(NT) void fork_kernel(ForkArgs a)
{
    __shared__ const uint8_t *sSrc[kMaxTileRows];
    const Shape &sh = a.sh;
    const int per_layer = a.host_tiles + a.hot_tiles + a.tail_tiles;
    const int64_t per_pair = 1 + (int64_t)per_layer * sh.n_layers;
    const int R = sh.R, C = a.ts.chunks;
    for (int64_t job = blockIdx.x; job < per_pair * a.n; job += gridDim.x) {
        const int i = (int)(job / per_pair);
        int64_t t = job - i * per_pair;
        const int32_t s = a.src[i], d = a.dst[i];
        bool bad = s < 0 || s >= sh.n_req || d < 0 || d >= sh.n_req;
        bad = bad || named_anywhere(a.src, a.n, d);
        bad = bad || named_earlier(a.dst, i, d) || named_anywhere(a.dst, a.n, s);
        if (t == 0) {
            if (!bad)
                fork_metadata(a, i, s, d);
            else if (threadIdx.x == 0 && a.status)
                a.status[i] = KVR_E_ARG;
            continue;
        }
        if (bad)
            continue;
        t -= 1;
        const LayerPtrs lp = a.layers[t / per_layer];
        t %= per_layer;
        const uint8_t *from;
        uint8_t *to;
        int64_t rows;
        int region = 0;  // 0 host, 1 hot, 2 tail
        if (t < a.host_tiles) {
            from = lp.host + (int64_t)s * sh.host_rows * R;
            to = lp.host + (int64_t)d * sh.host_rows * R;
            rows = a.m.L[s] < sh.host_rows ? a.m.L[s] : sh.host_rows;
        } else if (t < a.host_tiles + a.hot_tiles) {
            t -= a.host_tiles;
            region = 1;
            from = lp.hot + (int64_t)s * sh.B * R;
            to = lp.hot + (int64_t)d * sh.B * R;
            rows = sh.B;
        } else {
            t -= a.host_tiles + a.hot_tiles;
            region = 2;
            from = lp.tail + (int64_t)s * sh.T * R;
            to = lp.tail + (int64_t)d * sh.T * R;
            rows = sh.T;
        }
        const int64_t j0 = t * a.ts.rows;
        if (j0 >= rows)
            continue;
        const int nrows = (int)(rows - j0 < a.ts.rows ? rows - j0 : a.ts.rows);
        __syncthreads();  // the previous tile's readers are done with sSrc
        if ((int)threadIdx.x < nrows) {
            const int64_t row = j0 + threadIdx.x;
            const uint8_t *p = from + row * R;
            if (region == 0 && row < sh.H) {
                const int64_t e = (int64_t)s * sh.n_pages + row / sh.P;
                if (a.m.page_map[e] >= 0 || !a.m.host_valid[e])
                    p = nullptr;
            } else if (region == 1) {
                const int64_t b = (int64_t)s * sh.B + row;
                const int32_t pos = a.m.tag[b];
                if (pos < 0)
                    p = nullptr;
                else if (a.m.stamp[b] == a.m.clock[s] && host_copy(a, s, pos))
                    p = lp.host + ((int64_t)s * sh.host_rows + pos) * R;
            }
            sSrc[threadIdx.x] = p;
        }
        __syncthreads();
        const int total = nrows * C;
        uint8_t *out = to + j0 * R;
        for (int c0 = 0; c0 < total; c0 += NT * kUnroll) {
            u32x4 v[kUnroll];
            bool have[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int c = c0 + u * NT + threadIdx.x;
                have[u] = false;
                if (c < total) {
                    const int row = (int)(((uint64_t)(uint32_t)c * a.ts.magic) >> 32);
                    const uint8_t *p = sSrc[row];
                    if (p) {
                        have[u] = true;
                        load_chunk(v[u], p + (c - row * C) * 16);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (have[u])
                    store_chunk(out + (int64_t)(c0 + u * NT + threadIdx.x) * 16, v[u]);
        }
    }
}

// -------------------------------------------------------------- page moves

constexpr int kPartChunks = NT * kUnroll;  // 16-byte chunks a workgroup moves at once

// Workgroups that share a page, given how many jobs (pages times layers) there
// are at most: one if those fill the card, else up to one for each 32 KB.  (32
// pages of 73 KB, two layers, back to back: 13 us with one, 7 with three; the
// moves of a compaction of 256 such pages: 6 and 5 us.)
int page_parts(const Shape &sh, int64_t jobs)
{
    const int64_t most = ((int64_t)sh.P * sh.R / 16 + kPartChunks - 1) / kPartChunks;
    const int64_t want = kFullGrid / (jobs < 1 ? 1 : jobs);
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

// Part `part` of `parts` of a page of one layer within its pool, by the whole
// workgroup.
__device__ __forceinline__ void copy_page(const Shape &sh, uint8_t *pool, int32_t from, int32_t to,
                                          int part, int parts)
{
    const int64_t bytes = (int64_t)sh.P * sh.R;
    const int64_t chunks = bytes / 16;
    const uint8_t *src = pool + from * bytes;
    uint8_t *dst = pool + to * bytes;
    for (int64_t c0 = (int64_t)part * kPartChunks; c0 < chunks; c0 += (int64_t)parts * kPartChunks) {
        u32x4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + u * NT + threadIdx.x;
            if (c < chunks)
                load_chunk(v[u], src + c * 16);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + u * NT + threadIdx.x;
            if (c < chunks)
                store_chunk(dst + c * 16, v[u]);
        }
    }
}

struct CopyArgs {
    Shape sh;
    const LayerPtrs *layers;
    int32_t *page_map, *refs;
    const int32_t *req, *page, *phys;
    int32_t *status;
};

// grid (entries, layers, parts of a page).  Entries are judged on the state before the call:
// this launch writes no metadata, the commit launch after it does.
__global__ __launch_bounds__(NT) void copy_pages_kernel(CopyArgs a)
{
    const Shape &sh = a.sh;
    const int i = blockIdx.x;
    const int32_t r = a.req[i], p = a.page[i], ph = a.phys[i];
    int st = (r < 0 || r >= sh.n_req || p < 0 || p >= sh.H / sh.P) ? KVR_E_ARG : KVR_OK;
    bool repeat = false;
    for (int j = threadIdx.x; j < i; j += NT)
        repeat |= (a.req[j] == r && a.page[j] == p) || a.phys[j] == ph;
    if (__syncthreads_or(repeat) && st == KVR_OK)
        st = KVR_E_ARG;
    if (st == KVR_OK && !in_pool(sh, ph))
        st = KVR_E_RANGE;
    int32_t from = -1;
    if (st == KVR_OK) {
        from = a.page_map[(int64_t)r * sh.n_pages + p];
        if (!in_pool(sh, from) || a.refs[ph] > 0)
            st = KVR_E_STATE;
    }
    if (st == KVR_OK)
        copy_page(sh, a.layers[blockIdx.y].pool, from, ph, blockIdx.z, gridDim.z);
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        a.status[i] = st;
}

__global__ __launch_bounds__(NT) void copy_commit_kernel(CopyArgs a, int32_t n)
{
    const int i = blockIdx.x * NT + threadIdx.x;
    if (i >= n || a.status[i] != KVR_OK)
        return;
    int32_t *e = a.page_map + (int64_t)a.req[i] * a.sh.n_pages + a.page[i];
    atomicSub(&a.refs[*e], 1);
    atomicAdd(&a.refs[a.phys[i]], 1);
    *e = a.phys[i];
}

// ------------------------------------------------- free list and compaction
//
// Both need, for each page, the number of live pages below it.  The pool is
// cut into at most kPoolBlocks blocks; a first launch counts each block's live
// pages, and every block of the next adds up the counts before its own.  A
// pool of one block (up to 2048 pages) needs no first launch.

constexpr int kPoolBlocks = 1024;
constexpr int kPoolChunk = 2048;  // pages a workgroup looks at in one step
constexpr int kPoolItems = kPoolChunk / NT;

struct PoolArgs {
    int64_t pages;
    int32_t per_block, blocks;
    const int32_t *refs;
    int32_t *block_live;  // [blocks] workspace
    int32_t *rank;        // [pages] workspace (compaction)
    int32_t *free_list, *free_count;
    int32_t *moves, *move_count;  // [pages][2]: source, destination
    int32_t max_moves;
};

__global__ __launch_bounds__(NT) void count_live_kernel(PoolArgs a)
{
    const int64_t p0 = (int64_t)blockIdx.x * a.per_block;
    int live = 0;
    for (int64_t p = p0 + threadIdx.x; p < p0 + a.per_block && p < a.pages; p += NT)
        live += a.refs[p] > 0;
    __shared__ int sLive;
    if (threadIdx.x == 0)
        sLive = 0;
    __syncthreads();
    atomicAdd(&sLive, live);
    __syncthreads();
    if (threadIdx.x == 0) {
        a.block_live[blockIdx.x] = sLive;
        if (blockIdx.x == 0 && a.move_count)
            *a.move_count = 0;
    }
}

// Per page: free ones go to the free list in order (PLAN false), or pair the
// highest live pages with the lowest free ones (PLAN true).  With `live` live
// pages, page p >= live that is live moves, and its rank from the top is the
// number of live pages above it; page p < live that is free is filled, and
// its rank is the number of free pages below it.  Both kinds are equally
// many, so ranks pair them.
template <bool PLAN>
__global__ __launch_bounds__(NT) void rank_pages_kernel(PoolArgs a)
{
    __shared__ int sSum[2], sWave[kPoolItems][NT / 64], sMoved;
    if (threadIdx.x < 2)
        sSum[threadIdx.x] = 0;
    if (threadIdx.x == 0)
        sMoved = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t p0 = (int64_t)blockIdx.x * a.per_block;
    const int64_t p1 = p0 + a.per_block < a.pages ? p0 + a.per_block : a.pages;
    bool is[kPoolItems];
    auto load = [&](int64_t c) {
#pragma unroll
        for (int k = 0; k < kPoolItems; ++k) {
            const int64_t p = c + k * NT + threadIdx.x;
            is[k] = p < p1 && a.refs[p] > 0;
        }
    };
    load(p0);
    int before = 0, all = 0;
    if (a.blocks == 1) {
#pragma unroll
        for (int k = 0; k < kPoolItems; ++k)
            all += is[k];
    } else {
        for (int b = threadIdx.x; b < a.blocks; b += NT) {
            const int v = a.block_live[b];
            all += v;
            before += b < (int)blockIdx.x ? v : 0;
        }
    }
    __syncthreads();
    atomicAdd(&sSum[0], before);
    atomicAdd(&sSum[1], all);
    __syncthreads();
    int base = sSum[0];
    const int live = sSum[1];
    int moved = 0;
    for (int64_t c = p0; c < p1; c += kPoolChunk) {
        if (c > p0)
            load(c);
        uint64_t mask[kPoolItems];
#pragma unroll
        for (int k = 0; k < kPoolItems; ++k) {
            mask[k] = __ballot(is[k]);
            if (lane == 0)
                sWave[k][wave] = __popcll(mask[k]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPoolItems; ++k) {
            int below = base + __popcll(mask[k] & ((1ull << lane) - 1ull));
            for (int w = 0; w < NT / 64; ++w) {
                below += w < wave ? sWave[k][w] : 0;
                base += sWave[k][w];
            }
            const int64_t p = c + k * NT + threadIdx.x;
            if (p >= p1)
                continue;
            if (!PLAN) {
                if (!is[k])
                    a.free_list[p - below] = (int32_t)p;
                continue;
            }
            if (p >= live) {
                const int rank = live - 1 - below;
                const bool goes = is[k] && rank < a.max_moves;
                a.rank[p] = goes ? rank : -1;
                if (goes) {
                    a.moves[2 * (int64_t)rank] = (int32_t)p;
                    ++moved;
                }
            } else if (!is[k] && p - below < a.max_moves) {
                a.moves[2 * (p - below) + 1] = (int32_t)p;
            }
        }
        __syncthreads();  // sWave is rewritten by the next chunk
    }
    if (PLAN) {
        atomicAdd(&sMoved, moved);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (a.blocks == 1) {
                *a.move_count = sMoved;
                a.block_live[0] = live;
            } else if (sMoved) {
                atomicAdd(a.move_count, sMoved);
            }
        }
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.free_count = (int32_t)(a.pages - live);
    }
}

struct CompactArgs {
    Shape sh;
    const LayerPtrs *layers;
    int32_t *page_map, *refs;
    const int32_t *rank, *moves, *move_count, *block_live;
    int32_t blocks, map_blocks, parts;
};

// Workgroups [0, map_blocks) bring the page maps in line, the others move the
// pages (and their counts).  Sources lie above every destination and are not
// written, so the moves may run in any order.
__global__ __launch_bounds__(NT) void compact_kernel(CompactArgs a)
{
    const Shape &sh = a.sh;
    if ((int)blockIdx.x < a.map_blocks) {
        __shared__ int sLive;
        if (threadIdx.x == 0)
            sLive = 0;
        __syncthreads();
        int live = 0;
        for (int b = threadIdx.x; b < a.blocks; b += NT)
            live += a.block_live[b];
        atomicAdd(&sLive, live);
        __syncthreads();
        live = sLive;
        const int64_t n = (int64_t)sh.n_req * sh.n_pages;
        for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < n;
             e += (int64_t)a.map_blocks * NT) {
            const int32_t ph = a.page_map[e];
            if (!in_pool(sh, ph) || ph < live)
                continue;
            const int32_t k = a.rank[ph];
            if (k >= 0)
                a.page_map[e] = a.moves[2 * (int64_t)k + 1];
        }
        return;
    }
    const int moves = *a.move_count;
    const int per_move = sh.n_layers * a.parts;
    const int64_t jobs = (int64_t)moves * per_move;
    for (int64_t job = blockIdx.x - a.map_blocks; job < jobs; job += gridDim.x - a.map_blocks) {
        const int k = (int)(job / per_move), rest = (int)(job - (int64_t)k * per_move);
        const int l = rest / a.parts, part = rest - l * a.parts;
        const int32_t from = a.moves[2 * (int64_t)k], to = a.moves[2 * (int64_t)k + 1];
        copy_page(sh, a.layers[l].pool, from, to, part, a.parts);
        if (rest == 0 && threadIdx.x == 0) {
            a.refs[to] = a.refs[from];
            a.refs[from] = 0;
        }
    }
}

int64_t pool_pages(const kvr_ctx *c) { return c->shape.pool_rows / c->shape.P; }

PoolArgs pool_args(const kvr_ctx *c, void *workspace)
{
    PoolArgs a{};
    a.pages = pool_pages(c);
    const int64_t per = (a.pages + kPoolBlocks - 1) / kPoolBlocks;
    a.per_block = (int32_t)((per < 1 ? 1 : (per + kPoolChunk - 1) / kPoolChunk) * kPoolChunk);
    a.blocks = (int32_t)((a.pages + a.per_block - 1) / a.per_block);
    a.refs = c->page_refs;
    a.block_live = static_cast<int32_t *>(workspace);
    a.rank = a.block_live + kPoolBlocks;
    return a;
}

hipError_t launch_count_live(const kvr_ctx *c, const PoolArgs &a, hipStream_t s)
{
    if (a.blocks == 1)
        return hipSuccess;
    return launch(c, KVR_KERNEL_PAGES, count_live_kernel, dim3(a.blocks), dim3(NT), 0, s, a);
}

unsigned blocks_for(int64_t items, int64_t most)
{
    const int64_t b = (items + NT - 1) / NT;
    return (unsigned)(b < 1 ? 1 : (b > most ? most : b));
}

MetaPtrs meta_ptrs(const kvr_ctx *c)
{
    return MetaPtrs{c->L, c->page_map, c->host_valid, c->tag, c->stamp, c->clock, c->page_refs};
}

}  // namespace

size_t pool_workspace_bytes(const kvr_ctx *c)
{
    return sizeof(int32_t) * (size_t)(kPoolBlocks + pool_pages(c));
}

hipError_t launch_count_refs(const kvr_ctx *c, hipStream_t s)
{
    const int64_t pages = pool_pages(c);
    if (pages == 0)
        return hipSuccess;
    hipError_t e = launch(c, KVR_KERNEL_PAGES, zero_kernel, dim3(blocks_for(pages, 4096)), dim3(NT),
                          0, s, c->page_refs, pages);
    if (e != hipSuccess)
        return e;
    const int64_t entries = (int64_t)c->shape.n_req * c->shape.n_pages;
    return launch(c, KVR_KERNEL_PAGES, count_refs_kernel, dim3(blocks_for(entries, 4096)), dim3(NT),
                  0, s, c->shape, c->page_map, c->page_refs);
}

hipError_t launch_release(const kvr_ctx *c, int32_t n, const int32_t *ids, int32_t *status,
                          hipStream_t s)
{
    return launch(c, KVR_KERNEL_PAGES, release_kernel, dim3(n), dim3(NT), 0, s, c->shape,
                  meta_ptrs(c), ids, status);
}

hipError_t launch_fork(const kvr_ctx *c, int32_t n, const int32_t *src, const int32_t *dst,
                       int32_t *status, hipStream_t s)
{
    ForkArgs a{};
    a.sh = c->shape;
    a.m = meta_ptrs(c);
    a.ts = tile_for(c->shape, kUnroll);
    a.layers = c->layers_d;
    a.src = src;
    a.dst = dst;
    a.status = status;
    a.n = n;
    const int rows = a.ts.rows;
    a.host_tiles = (int32_t)((a.sh.host_rows + rows - 1) / rows);
    a.hot_tiles = (a.sh.B + rows - 1) / rows;
    a.tail_tiles = (a.sh.T + rows - 1) / rows;
    const int64_t jobs =
        n * (1 + (int64_t)(a.host_tiles + a.hot_tiles + a.tail_tiles) * a.sh.n_layers);
    return launch(c, KVR_KERNEL_PAGES, fork_kernel,
                  dim3((unsigned)(jobs < kMaxCopyBlocks ? jobs : kMaxCopyBlocks)), dim3(NT), 0, s, a);
}

hipError_t launch_copy_pages(const kvr_ctx *c, int32_t n, const int32_t *req, const int32_t *page,
                             const int32_t *phys, int32_t *status, hipStream_t s)
{
    CopyArgs a{c->shape, c->layers_d, c->page_map, c->page_refs, req, page, phys, status};
    const int parts = page_parts(c->shape, (int64_t)n * c->shape.n_layers);
    hipError_t e = launch(c, KVR_KERNEL_PAGES, copy_pages_kernel,
                          dim3(n, c->shape.n_layers, parts), dim3(NT), 0, s, a);
    if (e != hipSuccess)
        return e;
    return launch(c, KVR_KERNEL_PAGES, copy_commit_kernel, dim3((n + NT - 1) / NT), dim3(NT), 0, s,
                  a, n);
}

hipError_t launch_list_free(const kvr_ctx *c, int32_t *free_list, int32_t *free_count,
                            void *workspace, hipStream_t s)
{
    PoolArgs a = pool_args(c, workspace);
    a.free_list = free_list;
    a.free_count = free_count;
    if (a.pages == 0)
        return launch(c, KVR_KERNEL_PAGES, zero_kernel, dim3(1), dim3(NT), 0, s, free_count,
                      (int64_t)1);
    hipError_t e = launch_count_live(c, a, s);
    if (e != hipSuccess)
        return e;
    return launch(c, KVR_KERNEL_PAGES, rank_pages_kernel<false>, dim3(a.blocks), dim3(NT), 0, s, a);
}

hipError_t launch_compact(const kvr_ctx *c, int32_t max_moves, int32_t *moves, int32_t *move_count,
                          void *workspace, hipStream_t s)
{
    PoolArgs a = pool_args(c, workspace);
    a.moves = moves;
    a.move_count = move_count;
    a.max_moves = max_moves;
    if (a.pages == 0)
        return launch(c, KVR_KERNEL_PAGES, zero_kernel, dim3(1), dim3(NT), 0, s, move_count,
                      (int64_t)1);
    hipError_t e = launch_count_live(c, a, s);
    if (e != hipSuccess)
        return e;
    e = launch(c, KVR_KERNEL_PAGES, rank_pages_kernel<true>, dim3(a.blocks), dim3(NT), 0, s, a);
    if (e != hipSuccess)
        return e;
    CompactArgs k{c->shape, c->layers_d, c->page_map, c->page_refs, a.rank, moves, move_count,
                  a.block_live, a.blocks, 0, 1};
    k.map_blocks = (int32_t)blocks_for((int64_t)k.sh.n_req * k.sh.n_pages, 256);
    const int64_t pages = (a.pages / 2 < max_moves ? a.pages / 2 : max_moves) * k.sh.n_layers;
    k.parts = page_parts(k.sh, pages);
    const int64_t most = pages * k.parts;
    const int64_t copies = most < 1 ? 1 : (most > 8192 ? 8192 : most);
    return launch(c, KVR_KERNEL_PAGES, compact_kernel, dim3((unsigned)(k.map_blocks + copies)),
                  dim3(NT), 0, s, k);
}

}  // namespace kvr
