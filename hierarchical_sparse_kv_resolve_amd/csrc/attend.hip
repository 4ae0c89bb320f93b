// Attention of new tokens over resolved rows ("Adaptive DHiSparse:
// Speculative Decoding over a Load-Adaptive KV Hierarchy", section "How it
// works", paragraph "Model-specific reuse": attention consumes the rows that
// the location vector names).
//
// A row is one token's latent c (d_v values) and rope part r; its key is
// (c, r), its value c, shared by all heads.  For a query row x (a head of a
// query) over the rows j it attends to:
//   t_j = log2(e) * scale * (q . key_j),  p_j = 2^(t_j - m),  l = sum p_j,
//   out = sum p_j c_j / l,                lse = ln 2 * (m + log2 l)
// with one pass over the rows: m is a reference at most 8 below the running
// maximum (so p <= 2^8; fp16 rows: 6, and every p is raised by 2^9, see
// Mfma); when a tile exceeds it, it becomes the maximum and l and the sums are
// scaled down.
//
// A workgroup of NW waves owns MB blocks of 16 query rows and a share of the
// selection, which it walks in tiles of kTile (64) rows, kept in LDS.  Tiles arrive
// by 16-byte direct loads to LDS, addresses from the location words, which are
// read two tiles earlier still.
//   scores   a wave computes 16 of the tile's rows for one block of query rows
//            by 16x16x32 MFMA, the keys from LDS and the queries in registers;
//   values   every wave takes d_v / NW columns of all query rows; the
//            probabilities pass through LDS, the latents are read transposed
//            (ds_read_tr), so the product needs no copy of the tile.
// With three tiles in LDS the values of one are summed beside the scores of
// the next, while the one after is on its way, and a tile costs one barrier;
// with two (where three do not fit), its values follow its own scores.
// Both products leave a query row in one lane (mod 16), so the running
// maximum, the sums and their corrections stay in registers.
//
// 16-byte chunks of a row lie in LDS at chunk ^ swizzle(row): the 8 (keys) or
// 4 (latents) rows that a read touches at once are then in different banks.
// The permutation is applied to the source address of the direct loads.
//
// 8-bit rows stay 8-bit in LDS.  Codes are exact in bf16, so no product is
// rounded: the scores sum each 128-value group apart and weigh it with its
// scale, and the probabilities are multiplied by the row's scale of the
// columns' group before they are rounded to bf16.
//
// Rows left out are read from a row of zeros and their p is 0.
//
// What bounds it (one MI355X, calls over changing inputs; the kernel, then the
// join of the shares):
// with few query rows a selection, reading the rows,
//   64 requests x 16 heads x 2048 fp8 rows of 656 bytes     28 + 5 us, 3.1 TB/s
//   32 requests x 4 queries x 16 heads x 2048 bf16 rows of a union of 3277,
//   each query its own rows                        49 + 6 us, 6.1 TB/s read
//   (302 MB through the L2s, which miss 241 MB of it: twice the union's 121);
// with many, the vector, matrix and LDS instructions of two waves a SIMD,
//   64 requests x 128 heads x 2048 fp8 rows        77 us, 475 TFLOP/s
//   (0.40 of what a large bf16 product reaches): by its counters a tile takes
//   5000 cycles, of which a SIMD's vector instructions (exponentials, widened
//   codes, addresses) issue for 2550 and its matrix unit works for 1090, and
//   the LDS is busy for 1890, 580 of them bank conflicts; a wave waits for its
//   turn to issue in 26 % of its cycles and at barriers and counters in 35 %;
// with few rows in all, latency: one request x 16 heads x 256 rows takes
//   10 + 4 us (an empty kernel 4), four dependent loads (lists, words, rows)
//   and one tile.
//
// Split, block and buffers, each against the form of the kernel that it was
// tried on (128 heads as above, the present form then 75 us): scores split over
// the waves by dimension, two barriers a tile 89 us; 64 query rows and 8 waves
// 77 and a join of 9; 16 waves of 128 registers 110; 4 waves of 512 registers
// 92; two workgroups a compute unit 90; 32 query rows, 8 waves and tiles of 64
// rows 75 (taken).  Tiles of 32 rows took longer in blocks of 16 query rows too
// (the 16-head cases above 28 instead of 26 and 59 instead of 53 us then).
#include "block.h"
#include "kvr_internal.h"
#include "rowformat.h"

namespace kvr {
namespace {

constexpr int kTile = 64;     // rows per tile

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A workgroup barrier that leaves direct loads to LDS in flight (the next
// tile's), unlike __syncthreads.
__device__ __forceinline__ void barrier_lds()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The same once this wave's direct loads have arrived.
__device__ __forceinline__ void barrier_all()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Direct loads to LDS: lane i's 16 (or 4) bytes go to lds + 16 i (4 i).  They
// are written as assembly because the compiler, which cannot tell the two
// buffers of a tile apart, would otherwise wait for them before the next LDS
// read; the kernel waits itself (barrier_all) before it reads what they bring.
__device__ __forceinline__ uint32_t lds_offset(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

__device__ __forceinline__ void load_lds16(uint32_t lds, const void *src)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
                 : "memory", "m0");
}

__device__ __forceinline__ void load_lds4(uint32_t lds, const void *src)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
                 : "memory", "m0");
}

#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T *)(p))

// What a row that is left out is read from (the longest row is 1152 bytes).
__device__ __attribute__((aligned(16))) uint8_t zero_row[1152];
__device__ int32_t zero_words[4];

struct AttendArgs {
    Shape sh;
    const LayerPtrs *layers;  // device table
    kvr_attend_call c;
    int32_t units;      // selections: entries, or (entry, query) with a map
    int32_t unit_rows;  // query rows that share a selection
    int32_t groups;     // workgroups per selection and share
    int32_t shares;
    bool wide;          // q may be read 16 bytes at a time
    float *partial;     // [units][shares][unit_rows][d_v], with shares > 1
    float *stat;        // [units][shares][unit_rows][2]: m, l
};

// MFMA operands of a 16-bit type.  Probabilities are kept as 2^(t_j - m + kLift),
// and m is at most kSlack below the running maximum.  bf16 has the exponents of
// 32 bits and needs no lift.  fp16 ends at 2^16 and has steps of 2^-24, so its
// probabilities are raised to at most 2^15: the steps are then 2^-33 of the
// largest probability, and what 2^22 rows lose to them stays below 2^-12 of the
// largest value (2^24, the most a call takes: 2^-10).  Without the lift 2^18
// rows of weight 2^-25 each, a hundredth of the result together, were lost.
// (The ragged fp16 case: 19.2 us without a lift and slack 8, 19.2 with slack 6
// and lift 9, 20.3 with slack 4 and lift 11, where sums are scaled more often.)
template <typename E>
struct Mfma;
template <>
struct Mfma<__bf16> {
    static constexpr float kSlack = 8.f, kLift = 0.f;
    typedef __bf16 frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mul(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    static constexpr float kSlack = 6.f, kLift = 9.f;
    typedef _Float16 frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mul(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Swizzle of a row: bijective on any 8 consecutive rows, and different in its
// upper two bits on any 4 (a transposed 16-bit read takes pairs of chunks).
__device__ __forceinline__ constexpr int swizzle(int row)
{
    return ((row & 3) << 1) | ((row >> 2) & 1);
}

// 8 e4m3 codes as bf16 values.
__device__ __forceinline__ Mfma<__bf16>::frag widen(uint32_t lo, uint32_t hi)
{
    typedef Mfma<__bf16>::frag frag;
    frag f;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1];
    f[4] = c[0], f[5] = c[1], f[6] = d[0], f[7] = d[1];
    return f;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// The rows of one (entry, query) and where they are read.
struct RowList {
    const int32_t *map;   // this query's entries of the union, or null
    const uint32_t *loc;  // this entry's words, or null
    const uint8_t *tail, *pool, *hot;  // the request's places, or all the gathered rows
    bool gathered;
    int len;              // entries of the list
    int count;            // entries of the selection
};

// Address of the row of word w (entry e of the selection, -1: none), or null
// when it is left out; bad: w lies outside its place.  Selects only, so that
// it is scheduled among the products.
__device__ __forceinline__ const uint8_t *row_address(const Shape &sh, const RowList &list, int e,
                                                      uint32_t w, bool &bad)
{
    const bool in = e >= 0 && w != KVR_LOC_INVALID;
    const uint32_t place = w >> kPlaceShift;
    const bool tail = place == KVR_PLACE_TAIL, page = place == KVR_PLACE_PAGE;
    const uint32_t at = w & (place == KVR_PLACE_HOT ? kSlotMask : kIndexMask);
    const uint32_t limit = tail ? (uint32_t)sh.T : page ? (uint32_t)sh.pool_rows : (uint32_t)sh.B;
    // (opaque, so that the choice is made between registers)
    const uint8_t *at_tail = list.tail, *at_page = list.pool, *at_hot = list.hot;
    asm("" : "+s"(at_tail), "+s"(at_page), "+s"(at_hot));
    const uint8_t *base = tail ? at_tail : page ? at_page : at_hot;
    const bool ok = list.gathered || (place != KVR_PLACE_INVALID && at < limit);
    const uint32_t idx = list.gathered ? (uint32_t)e : at;
    bad = in && !ok;
    return in && ok ? base + (uint64_t)idx * (uint32_t)sh.R : nullptr;
}

// A tile in LDS: latents, rope parts and (8-bit rows) scales, each part
// [kTile rows][its bytes].
template <int FMT, int DV, int DR>
struct Tile {
    static constexpr bool kFp8 = FMT == KVR_ROW_FP8;
    static constexpr int kLatent = kFp8 ? DV : 2 * DV;  // bytes of a row's parts
    static constexpr int kRope = 2 * DR;
    static constexpr int kScales = kFp8 ? scale_bytes(DV) : 0;
    static constexpr int kRopeAt = kTile * kLatent;
    static constexpr int kScalesAt = kRopeAt + kTile * kRope;
    static constexpr int kBytes = kScalesAt + kTile * kScales;

    // The direct loads of ROWS rows, each of up to 1024 consecutive bytes of a
    // part in LDS.
    template <int ROWS>
    struct Loads {
        static constexpr int kLatentRows = 1024 / kLatent < ROWS ? 1024 / kLatent : ROWS;
        static constexpr int kRopeRows = DR == 0 ? ROWS : 1024 / kRope < ROWS ? 1024 / kRope : ROWS;
        static constexpr int kLatentLoads = ROWS / kLatentRows;
        static constexpr int kRopeLoads = DR == 0 ? 0 : ROWS / kRopeRows;
        const uint8_t *src[kLatentLoads + kRopeLoads + (kFp8 ? 1 : 0)];

        // Lane i < ROWS holds the address of row first + i of the tile.
        __device__ __forceinline__ void prepare(int first, const uint8_t *row)
        {
            const int lane = lane_id();
            const uint32_t lo = (uint32_t)(uintptr_t)row, hi = (uint32_t)((uintptr_t)row >> 32);
            auto source = [&](int k, int chunks, int from) __attribute__((always_inline)) {
                // (a 32-bit offset and its carry: one register each for the
                // offsets the compiler keeps)
                const uint32_t off = from + ((lane % chunks) ^ swizzle(first + k)) * 16;
                const uint32_t l = (uint32_t)__shfl((int)lo, k) + off;
                const uint32_t h = (uint32_t)__shfl((int)hi, k) + (l < off);
                return reinterpret_cast<const uint8_t *>((uint64_t)h << 32 | l);
            };
#pragma unroll
            for (int i = 0; i < kLatentLoads; ++i)
                src[i] = source(i * kLatentRows + lane / (kLatent / 16), kLatent / 16, 0);
#pragma unroll
            for (int i = 0; i < kRopeLoads; ++i)
                src[kLatentLoads + i] =
                    source(i * kRopeRows + lane / (kRope / 16), kRope / 16, kLatent + kScales);
            if constexpr (kFp8)
                src[kLatentLoads + kRopeLoads] = row + kLatent;
        }

        static constexpr int kCount = kLatentLoads + kRopeLoads + (kFp8 ? 1 : 0);
        // Starts load n, into the tile at LDS offset `lds`.
        __device__ __forceinline__ void start(int n, uint32_t lds, int first) const
        {
            const int lane = lane_id();
            if (n < kLatentLoads) {
                if (kLatentRows * kLatent == 1024 || lane < kLatentRows * kLatent / 16)
                    load_lds16(lds + (first + n * kLatentRows) * kLatent, src[n]);
            } else if (n < kLatentLoads + kRopeLoads) {
                const int i = n - kLatentLoads;
                if (kRopeRows * kRope == 1024 || lane < kRopeRows * kRope / 16)
                    load_lds16(lds + kRopeAt + (first + i * kRopeRows) * kRope, src[n]);
            } else if (lane < ROWS) {
                load_lds16(lds + kScalesAt + first * 16, src[n]);
            }
        }
    };
};

template <int FMT, int DV, int DR, int MB, int BUFS>
__global__ __launch_bounds__(MB * kTile * 4) void attend_kernel(AttendArgs a)
{
    typedef typename Elem<FMT>::type E;
    typedef Mfma<E> M;
    typedef typename M::frag frag;
    typedef E e4 __attribute__((ext_vector_type(4)));
    typedef Tile<FMT, DV, DR> TL;
    constexpr bool kFp8 = FMT == KVR_ROW_FP8;
    constexpr int kSteps = (DV + DR) / 32;    // MFMA steps of a score
    constexpr int RG = kTile / 16;             // row blocks of a tile
    constexpr int NW = MB * RG;               // waves: a block of scores each
    constexpr int NC = DV / NW / 16;          // value column blocks of a wave
    constexpr int kGroups = kFp8 ? DV / kScaleGroup : 1;
    constexpr int kRows = kTile / NW;          // rows a wave loads
    static_assert(DV % (NW * 16) == 0 && kRows >= 4 && kRows <= 16, "");

    __shared__ __attribute__((aligned(1024))) uint8_t sTile[BUFS * TL::kBytes];
    __shared__ __attribute__((aligned(16))) E sP[BUFS - 1][kGroups][MB * 16][kTile];
    __shared__ float sMax[RG][MB * 16];
    __shared__ uint16_t sValid[2][NW];
    __shared__ int sExceeds[4];  // whether a tile's probabilities must be written again
    __shared__ uint32_t sWord[2][kTile];  // location words, and with a map the
    __shared__ int32_t sEntry[2][kTile];  // entries, of tiles to come

    const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int rg = wave % RG, hg = wave / RG;  // the wave's block of scores

    // Workgroups are dealt to the 8 XCDs in turn: each XCD takes a run of
    // neighbours, so that its L2 serves the rows of one selection and share to
    // all their blocks, and those of a verification block to its queries.
    // (With selections and shares dealt to the XCDs in turn instead, the verify
    // block above took 54 us instead of 51, and one request of 64 x 128 query
    // rows, which then ran on one XCD, 543 instead of 76.)
    const uint32_t total = (uint32_t)(a.units * a.shares) * (uint32_t)a.groups;
    const uint32_t job = (blockIdx.x & 7) * ((total + 7) / 8) + blockIdx.x / 8;
    if (job >= total)
        return;
    const uint32_t us = job / (uint32_t)a.groups;
    const int g = (int)(job - us * (uint32_t)a.groups);
    const int unit = (int)(us / (uint32_t)a.shares), share = (int)us - unit * a.shares;
    const int i = a.c.map ? unit / a.c.nq : unit;
    // The loads that the rows' addresses depend on are issued together (what is
    // not given is read from the zeros), so that their latencies overlap.
    const int32_t *req_ids = a.c.req_ids ? a.c.req_ids + i : zero_words;
    const int32_t *counts = a.c.count ? a.c.count + i : zero_words;
    const int32_t req_read = *req_ids, count_read = *counts;
    const LayerPtrs lp = a.layers[a.c.layer];
    const int r = a.c.req_ids ? req_read : i;
    const bool known = r >= 0 && r < a.sh.n_req;

    RowList list;
    int cnt = a.c.count ? count_read : a.c.stride;
    list.count = known ? (cnt < 0 ? 0 : (cnt > a.c.stride ? a.c.stride : cnt)) : 0;
    list.len = a.c.map && list.count > 0 ? a.c.k : list.count;
    list.map = a.c.map ? a.c.map + (int64_t)unit * a.c.k : nullptr;
    list.loc = a.c.loc ? a.c.loc + (int64_t)i * a.c.stride : nullptr;
    list.gathered = a.c.rows != nullptr;
    if (!known && a.c.status && threadIdx.x == 0)
        a.c.status[i] = KVR_E_ARG;
    if (list.gathered) {
        list.tail = list.pool = list.hot =
            static_cast<const uint8_t *>(a.c.rows) + (int64_t)i * a.c.stride * a.sh.R;
    } else {
        list.tail = lp.tail + (int64_t)r * a.sh.T * a.sh.R;
        list.pool = lp.pool;
        list.hot = lp.hot + (int64_t)r * a.sh.B * a.sh.R;
    }

    const int tiles = (list.len + kTile - 1) / kTile;
    const int per = (tiles + a.shares - 1) / a.shares;
    const int t0 = share * per;
    const int t1 = t0 + per < tiles ? t0 + per : tiles;

    // query row x of the unit: query x / heads, head x % heads (with a map the
    // unit is one query)
    const E *q = static_cast<const E *>(a.c.q) + (int64_t)i * a.c.q_stride_entry;
    const int x0 = g * (MB * 16);
    frag qf[kSteps];  // of the wave's block (past the last query row: that row's,
                      // whose results are not written)
    auto load_q = [&](auto read) {
        const int x = x0 + hg * 16 + col;
        const int xc = x < a.unit_rows ? x : a.unit_rows - 1;
        const int qi = a.c.map ? unit % a.c.nq : xc / a.c.heads;
        const int h = a.c.map ? xc : xc % a.c.heads;
        const E *p = q + (int64_t)qi * a.c.q_stride_query + (int64_t)h * a.c.q_stride_head;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            // an 8-bit key fragment holds 8 of the 16 codes of one LDS read
            qf[s] = read(p + (kFp8 && s < DV / 32 ? s / 2 * 64 + grp * 16 + (s & 1) * 8
                                                  : s * 32 + grp * 8));
    };
    // m: the reference of this lane's query row in each block; m_own, l: that
    // of the wave's block and this lane's share of its sum
    float m[MB], m_own = -__builtin_inff(), l = 0.f;
    f32x4 o[NC][MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        m[mb] = -__builtin_inff();
#pragma unroll
        for (int c = 0; c < NC; ++c)
            o[c][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (threadIdx.x < 3)
        sExceeds[threadIdx.x] = 0;

    // This lane's row of a tile (a wave's first kRows lanes; the others repeat
    // them).  Its entry of the selection (-1: left out), its location word, its
    // address; a row past the list's end reads the last entry's.
    const int mine = wave * kRows + (lane & (kRows - 1));
    auto at = [&](int t) {
        const int j = t * kTile + mine;
        return j < list.len ? j : list.len - 1;
    };
    auto entry = [&](int t, int mapped) {
        const int e = list.map ? mapped : t * kTile + mine;
        return t < t1 && t * kTile + mine < list.len && e >= 0 && e < list.count ? e : -1;
    };
    const uint8_t *zeros = zero_row;
    asm volatile("" : "+s"(zeros));  // kept, not looked up for each tile
    typename TL::template Loads<kRows> loads;  // of the tile fetched next
    uint64_t valid = 0;                        // and which of its rows count
    bool any_bad = false;
    auto prepare = [&](int e, uint32_t w) __attribute__((always_inline)) {
        bool bad;
        const uint8_t *p = row_address(a.sh, list, e, w, bad);
        any_bad |= bad;
        valid = __ballot(p != nullptr);
        loads.prepare(wave * kRows, p ? p : zeros);
    };
    // Words and entries that are not given are read as 0.
    const uint32_t *loc = list.loc ? list.loc : reinterpret_cast<const uint32_t *>(zeros);
    const int32_t *map = list.map ? list.map : reinterpret_cast<const int32_t *>(zeros);
    auto word_at = [&](int e) { return loc + (list.loc && e >= 0 ? e : 0); };
    auto entry_at = [&](int t) { return map + (list.map ? at(t) : 0); };
    // Starts part `part` of `parts` of a tile's loads into a buffer.
    const uint32_t tiles_at = lds_offset(sTile);
    auto fetch = [&](int buf, int t, int part, int parts) __attribute__((always_inline)) {
        constexpr int N = TL::template Loads<kRows>::kCount;
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n * parts / N == part)
                loads.start(n, tiles_at + buf, wave * kRows);
        if (part == 0)
            sValid[t & 1][wave] = (uint16_t)(valid & ((1 << kRows) - 1));
    };

    const float to_log2 = a.c.scale * 1.44269504088896340736f;
    f32x4 s;    // t_j of the wave's block
    float sum;  // and the sum of its probabilities

    // (buf: where a tile lies in sTile)
    // LDS reads are issued in batches ahead of the products that use them
    // (sched_barrier keeps them there: left alone, each read is moved next to
    // its use and waited for).
    f32x4 w[kFp8 ? 4 : 1];  // scales of this lane's 4 rows of the block
    constexpr int kReads = TL::kLatent / 64;  // 16-byte reads of a key's latent
    constexpr int kBatch = kFp8 ? 2 : 4;      // of them at once: a scale group, or 4 steps
    constexpr int kBatches = kReads / kBatch;
    struct Keys {
        frag rope[DR > 0 ? DR / 32 : 1];
        u32x4 latent[2][kBatch];
    };
    const int kchunk[2] = {(grp ^ swizzle(col)) * 16, ((4 + grp) ^ swizzle(col)) * 16};
    auto read_keys = [&](Keys &key, int buf, int b) __attribute__((always_inline)) {
        const uint8_t *cur = sTile + buf;
        const int row = rg * 16 + col;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int n = b * kBatch + j;
            key.latent[b & 1][j] = *reinterpret_cast<const u32x4 *>(cur + row * TL::kLatent +
                                                                    kchunk[n & 1] + n / 2 * 128);
        }
        if (b > 0)
            return;
        if constexpr (DR > 0)
#pragma unroll
            for (int st = 0; st < DR / 32; ++st)
                key.rope[st] = *reinterpret_cast<const frag *>(
                    cur + TL::kRopeAt + row * TL::kRope + kchunk[st & 1] + st / 2 * 128);
        if constexpr (kFp8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = *reinterpret_cast<const f32x4 *>(cur + TL::kScalesAt +
                                                        (rg * 16 + grp * 4 + k) * 16);
    };
    // Scores of the wave's block of a tile whose first keys are being read;
    // then(b) starts what else is read or loaded beside batch b.
    auto scores = [&](Keys &key, int buf, auto then) __attribute__((always_inline)) {
        f32x4 even = {}, odd = {};
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
            if (b + 1 < kBatches)
                read_keys(key, buf, b + 1);
            then(b);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (kFp8) {
                f32x4 part = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 v = key.latent[b & 1][h];
                    part = M::mul(widen(v[0], v[1]), qf[b * 4 + h * 2], part);
                    part = M::mul(widen(v[2], v[3]), qf[b * 4 + h * 2 + 1], part);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    even[k] = fmaf(part[k], w[k][b], even[k]);
            } else {
#pragma unroll
                for (int j = 0; j < kBatch; j += 2) {
                    even = M::mul(__builtin_bit_cast(frag, key.latent[b & 1][j]),
                                  qf[b * kBatch + j], even);
                    odd = M::mul(__builtin_bit_cast(frag, key.latent[b & 1][j + 1]),
                                 qf[b * kBatch + j + 1], odd);
                }
            }
            if (b == 0 && DR > 0)
#pragma unroll
                for (int st = 0; st < DR / 32; ++st)
                    odd = M::mul(key.rope[st], qf[DV / 32 + st], odd);
        }
        s = even + odd;
    };

    // Probabilities of the wave's block of tile t, into LDS, rounded to the 16
    // bits that the matrix instructions take (off by at most 2^-8 of each for
    // bf16, 2^-11 for fp16 or 2^-34 of the largest; their sum l is taken before
    // the rounding).
    auto pchunk = [&](int head, int chunk) {  // 8 rows of a query row, swizzled
        return (chunk ^ (head & 7)) * 8;
    };
    auto write_p = [&](int t, const f32x4 *w) __attribute__((always_inline)) {
        const int pb = BUFS == 3 ? t & 1 : 0;
        const float ref = m_own == -__builtin_inff() ? 0.f : m_own - M::kLift;
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[k] = exp2_hw(s[k] - ref);
        sum = (p[0] + p[1]) + (p[2] + p[3]);
        const int head = hg * 16 + col;
        const int at = pchunk(head, rg * 2 + (grp >> 1)) + (grp & 1) * 4;
#pragma unroll
        for (int gi = 0; gi < kGroups; ++gi) {
            e4 v;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (kFp8)
                    v[k] = (E)(p[k] * w[k][gi]);
                else
                    v[k] = (E)p[k];
            }
            *reinterpret_cast<e4 *>(&sP[pb][gi][head][at]) = v;
        }
    };

    auto softmax = [&](int t, int flag) __attribute__((always_inline)) {
        const int first = rg * 16 + grp * 4;
        const uint32_t counts = sValid[t & 1][first / kRows] >> (first % kRows);
        bool exceeds = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s[k] = (counts >> k) & 1 ? s[k] * to_log2 : -__builtin_inff();
            exceeds |= s[k] > m_own + M::kSlack;
        }
        sExceeds[__any(exceeds) ? flag : 3] = 1;
        write_p(t, w);
    };

    // Tile t's probabilities are in LDS and one exceeded its reference: the
    // maximum becomes the reference, the sums so far are scaled down and the
    // tile's probabilities written again.
    auto settle = [&](int buf, int t) __attribute__((always_inline)) {
        float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (grp == 0)
            sMax[rg][hg * 16 + col] = top;
        barrier_lds();
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            float to = m[mb];
#pragma unroll
            for (int k = 0; k < RG; ++k)
                to = fmaxf(to, sMax[k][mb * 16 + col]);
            const float alpha = to == -__builtin_inff() ? 1.f : exp2_hw(m[mb] - to);
            m[mb] = to;
            m_own = hg == mb ? to : m_own;
            l = hg == mb ? l * alpha : l;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                o[c][mb] *= alpha;
        }
        f32x4 sc[kFp8 ? 4 : 1];  // the tile's scales once more
        if constexpr (kFp8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sc[k] = *reinterpret_cast<const f32x4 *>(sTile + buf + TL::kScalesAt +
                                                         (rg * 16 + grp * 4 + k) * 16);
        write_p(t, sc);
        barrier_lds();
    };

    // o[column][query row] += latent[row][column] * p[query row][row] of tile t:
    // its operands, then the products.
    struct Operands {
        frag p[kTile / 32][MB];
        i32x2 v[kTile / 32][NC][kFp8 ? 1 : 2];
    };
    const int gi_own = kFp8 ? wave * (DV / NW) / kScaleGroup : 0;
    auto read_p = [&](Operands &op, int t) __attribute__((always_inline)) {
        const int pb = BUFS == 3 ? t & 1 : 0;
#pragma unroll
        for (int st = 0; st < kTile / 32; ++st)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                op.p[st][mb] = *reinterpret_cast<const frag *>(
                    &sP[pb][gi_own][mb * 16 + col][pchunk(mb * 16 + col, st * 4 + grp)]);
    };
    auto read_v = [&](Operands &op, int buf) __attribute__((always_inline)) {
        const uint8_t *cur = sTile + buf;
#pragma unroll
        for (int st = 0; st < kTile / 32; ++st) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int cb = wave * NC + c;  // block of 16 columns
                if constexpr (kFp8) {
                    const int row = st * 32 + grp * 8 + (col >> 1);
                    op.v[st][c][0] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(LDS_PTR(
                        i32x2, cur + row * TL::kLatent + (cb ^ swizzle(row)) * 16 + (col & 1) * 8));
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = st * 32 + grp * 8 + h * 4 + (col >> 2);
                        const int chunk = (cb * 2 + ((col >> 1) & 1)) ^ swizzle(row);
                        op.v[st][c][h] = __builtin_bit_cast(
                            i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(
                                       s16x4, cur + row * TL::kLatent + chunk * 16 + (col & 1) * 8)));
                    }
                }
            }
        }
    };
    auto values = [&](const Operands &op) __attribute__((always_inline)) {
#pragma unroll
        for (int st = 0; st < kTile / 32; ++st) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                frag vf;
                if constexpr (kFp8)
                    vf = widen((uint32_t)op.v[st][c][0][0], (uint32_t)op.v[st][c][0][1]);
                else
                    vf = __builtin_bit_cast(frag, __builtin_shufflevector(op.v[st][c][0],
                                                                          op.v[st][c][kFp8 ? 0 : 1],
                                                                          0, 1, 2, 3));
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                    o[c][mb] = M::mul(vf, op.p[st][mb], o[c][mb]);
            }
        }
    };

    if (t0 < t1) {
        // the entries, words and addresses of the first tiles
        int mapped[4] = {};
        if (list.map)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mapped[k] = list.map[at(t0 + k)];
        const int e0 = entry(t0, mapped[0]), e1 = entry(t0 + 1, mapped[1]);
        int e = entry(t0 + 2, mapped[2]);
        uint32_t w0 = 0, w1 = 0, word = 0;
        if (list.loc) {
            w0 = list.loc[e0 < 0 ? 0 : e0];
            w1 = list.loc[e1 < 0 ? 0 : e1];
            word = list.loc[e < 0 ? 0 : e];
        }
        // the roles of the buffers and of the flags
        int prev = (BUFS - 1) * TL::kBytes, cur = 0, next = TL::kBytes;
        int f_prev = 2, f_cur = 0, f_next = 1;
        prepare(e0, w0);
        fetch(cur, t0, 0, 1);
        if (a.wide)
            load_q([](const E *p) { return *reinterpret_cast<const frag *>(p); });
        else
            load_q([](const E *p) {
                frag f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = p[e];
                return f;
            });
        prepare(e1, w1);
        if (lane < kRows) {
            sEntry[(t0 + 3) & 1][mine] = mapped[3];
            sWord[t0 & 1][mine] = word;
        }
        // On their way from tile t's turn: the rows of tile t + 1, the words of
        // tile t + 3, the map's entries of tile t + 4.  (Past the last tile they
        // are rows of zeros and repeated words.)
        int e3 = -1;
        auto ahead = [&](int t) __attribute__((always_inline)) {
            e3 = entry(t + 3, sEntry[(t + 3) & 1][mine]);
            if (lane < kRows) {
                load_lds4(lds_offset(&sWord[(t + 3) & 1][wave * kRows]), word_at(e3));
                load_lds4(lds_offset(&sEntry[t & 1][wave * kRows]), entry_at(t + 4));
            }
        };
        auto turn = [&]() __attribute__((always_inline)) {
            e = e3;
            const int free = prev, f_free = f_prev;
            prev = cur, cur = next, next = BUFS == 3 ? free : prev;
            f_prev = f_cur, f_cur = f_next, f_next = f_free;
        };
        Keys key;
        Operands op;
        int t = t0;
        uint32_t w2;
        // A tile up to its probabilities; three buffers: beside the values of
        // the tile before (but for the first).
        auto step = [&](auto first) __attribute__((always_inline)) {
            read_keys(key, cur, 0);
            w2 = sWord[t & 1][mine];
            __builtin_amdgcn_sched_barrier(0);
            sExceeds[f_next] = 0;  // set after the next barrier, read before this one
            ahead(t);
            scores(key, cur, [&](int b) __attribute__((always_inline)) {
                fetch(next, t + 1, b, kBatches);
                if (BUFS == 3 && !decltype(first)::value && b == kBatches - 1) {
                    read_p(op, t - 1);
                    read_v(op, prev);
                }
            });
            if (BUFS == 3 && !decltype(first)::value)
                values(op);
            softmax(t, f_cur);
            if (BUFS == 3) {
                prepare(e, w2);
                turn();
                ++t;
                barrier_all();
            } else {
                read_v(op, cur);
                barrier_lds();
            }
            return __builtin_amdgcn_readfirstlane(sExceeds[BUFS == 3 ? f_prev : f_cur]);
        };
        // Three buffers: after a step, t is the tile that has arrived, and tile
        // t - 1 has its probabilities in LDS.  Two: tile t has them.
        barrier_all();
        step(std::true_type());
        // The sums are scaled down (as they always are after the first tile)
        // between runs of tiles that stay below their references, not on a
        // branch inside the loop: there the compiler would keep two copies of
        // them (512 registers did not hold 128 of them twice).
        for (bool again = true; again;) {
            settle(BUFS == 3 ? prev : cur, BUFS == 3 ? t - 1 : t);
            again = false;
            for (;;) {
                l += sum;
                if (BUFS == 2) {
                    read_p(op, t);
                    values(op);
                    prepare(e, w2);
                    turn();
                    ++t;
                }
                if (t >= t1)
                    break;
                if (BUFS == 2)
                    barrier_all();
                if (step(std::false_type())) {
                    again = true;
                    break;
                }
            }
        }
        if (BUFS == 3) {
            read_p(op, t1 - 1);
            read_v(op, prev);
            values(op);
        }
    }
    if (any_bad && a.c.status)
        a.c.status[i] = KVR_E_RANGE;

    // the sums of the waves and lane groups that share a query row
    barrier_all();  // also: no load is on its way to LDS when the wave ends
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (grp == 0)
        sMax[rg][hg * 16 + col] = l;
    barrier_lds();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int x = x0 + mb * 16 + col;
        if (x >= a.unit_rows)
            continue;
        float sum = 0.f;  // of the query row
#pragma unroll
        for (int k = 0; k < RG; ++k)
            sum += sMax[k][mb * 16 + col];
        const int64_t at = (int64_t)unit * a.unit_rows + x;  // query row of the call
        const int c0 = wave * (DV / NW) + grp * 4;
        if (a.shares > 1) {
            const int64_t ps = (int64_t)us * a.unit_rows + x;
            if (wave == 0 && grp == 0)
                *reinterpret_cast<float2 *>(a.stat + 2 * ps) = make_float2(m[mb] - M::kLift, sum);
            if (m[mb] == -__builtin_inff() && sum == 0.f)
                continue;  // an empty share: its sums are not read
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<f32x4 *>(a.partial + ps * DV + c0 + c * 16) = o[c][mb];
            continue;
        }
        const float inv = m[mb] == -__builtin_inff() && sum == 0.f ? 0.f : 1.f / sum;
        if (wave == 0 && grp == 0 && a.c.lse)
            a.c.lse[at] = 0.69314718055994530942f * (m[mb] - M::kLift + __log2f(sum));
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            typedef E e4 __attribute__((ext_vector_type(4)));
            e4 v;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = (E)(o[c][mb][k] * inv);
            *reinterpret_cast<e4 *>(static_cast<E *>(a.c.out) + at * DV + c0 + c * 16) = v;
        }
    }
}

// Joins the shares of each query row: a workgroup per row, its waves taking
// every fourth share with several in flight, their sums added in wave order.
// Bound by the latency of reading them: 16 shares of 512 query rows (17 MB) in
// 5.3 us, of which an empty launch is 4, 32 shares in 9.0; one wave a row that
// reads one share after the other took 9.0 and 16.4.
constexpr int kJoinWaves = 4;
template <typename E, int DV>
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(AttendArgs a)
{
    constexpr int N = DV / 64;   // columns of a lane
    constexpr int kFlight = 4;   // shares in flight
    typedef float vec __attribute__((ext_vector_type(N)));
    __shared__ float sL[kJoinWaves];
    __shared__ vec sO[kJoinWaves][64];
    const int lane = lane_id(), wave = wave_id();
    const int64_t at = blockIdx.x;
    const int unit = (int)(at / a.unit_rows), x = (int)(at % a.unit_rows);
    const int64_t first = (int64_t)unit * a.shares * a.unit_rows + x;
    auto stat = [&](int s) {
        return *reinterpret_cast<const float2 *>(a.stat + 2 * (first + (int64_t)s * a.unit_rows));
    };
    float m = -__builtin_inff();
    for (int s = lane; s < a.shares; s += 64)
        m = fmaxf(m, stat(s).x);
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1)
        m = fmaxf(m, __shfl_xor(m, k));
    float l = 0.f;
    vec o = {};
    for (int s0 = wave; s0 < a.shares; s0 += kJoinWaves * kFlight) {
        vec part[kFlight];
        float w[kFlight], ls[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int s = s0 + f * kJoinWaves;
            w[f] = 0.f;
            ls[f] = 0.f;
            part[f] = vec{};
            if (s >= a.shares)
                continue;
            const float2 st = stat(s);
            if (st.x == -__builtin_inff() && st.y == 0.f)
                continue;  // an empty share: its sums were not written
            w[f] = st.x == -__builtin_inff() ? 1.f : exp2_hw(st.x - m);
            ls[f] = st.y;
            part[f] = *reinterpret_cast<const vec *>(
                a.partial + (first + (int64_t)s * a.unit_rows) * DV + lane * N);
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            l += w[f] * ls[f];
            o += w[f] * part[f];
        }
    }
    sO[wave][lane] = o;
    if (lane == 0)
        sL[wave] = l;
    __syncthreads();
    if (wave != 0)
        return;
#pragma unroll
    for (int k = 1; k < kJoinWaves; ++k) {
        l += sL[k];
        o += sO[k][lane];
    }
    const float inv = m == -__builtin_inff() && l == 0.f ? 0.f : 1.f / l;
    typedef E out __attribute__((ext_vector_type(N)));
    out v;
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = (E)(o[k] * inv);
    *reinterpret_cast<out *>(static_cast<E *>(a.c.out) + at * DV + lane * N) = v;
    if (lane == 0 && a.c.lse)
        a.c.lse[at] = 0.69314718055994530942f * (m + __log2f(l));
}

template <int FMT, int DV, int DR>
hipError_t launch_dims(const kvr_ctx *c, const AttendArgs &a, int block, dim3 grid, hipStream_t s)
{
    // Three tiles where LDS holds them (64 16-bit rows of 576 values are 72 KB):
    // 64 requests of 128 heads, fp8 rows, took 75 us with three, 79 with two.
    constexpr int kBufs = FMT == KVR_ROW_FP8 || DV == 256 ? 3 : 2;
    if (block == 16)
        return launch(c, KVR_KERNEL_ATTEND, attend_kernel<FMT, DV, DR, 1, kBufs>, grid,
                      dim3(256), 0, s, a);
    return launch(c, KVR_KERNEL_ATTEND, attend_kernel<FMT, DV, DR, 2, kBufs>, grid, dim3(512), 0,
                  s, a);
}

template <int FMT>
hipError_t launch_format(const kvr_ctx *c, const AttendArgs &a, int block, dim3 grid, hipStream_t s)
{
    if (a.c.d_v == 512)
        return a.c.d_rope ? launch_dims<FMT, 512, 64>(c, a, block, grid, s)
                          : launch_dims<FMT, 512, 0>(c, a, block, grid, s);
    return a.c.d_rope ? launch_dims<FMT, 256, 64>(c, a, block, grid, s)
                      : launch_dims<FMT, 256, 0>(c, a, block, grid, s);
}

template <typename E, int DV>
hipError_t launch_join(const kvr_ctx *c, const AttendArgs &a, hipStream_t s)
{
    return launch(c, KVR_KERNEL_ATTEND, join_kernel<E, DV>,
                  dim3((unsigned)((int64_t)a.units * a.unit_rows)), dim3(kJoinWaves * 64), 0, s, a);
}

constexpr int64_t kWorkgroups = 256;  // compute units: one workgroup each
constexpr int kMaxBlock = 32;         // query rows

int64_t partial_bytes(int64_t rows, int32_t d_v) { return rows * (d_v + 2) * (int64_t)sizeof(float); }

}  // namespace

// A selection shared by unit_rows query rows is cut into blocks of 16 or 32 of
// them, and into shares (of at least one tile) until every compute unit has a
// workgroup.
//   block   16 when that holds all the rows, else 32, which reads each tile half
//           as often: 64 requests of 128 heads 76 us against 124 in blocks of
//           16; 64 requests of 16 heads 27 us in either.  (8 requests of 64
//           heads over 16-bit rows do better in blocks of 16 with half as many
//           shares: 19 + 4 us instead of 21 + 5.)
//   shares  256 workgroups (kernel + join): 8 requests of 64 heads, 2048 rows
//           with 128 of them 22 + 4 us, with 256 21 + 5, with 512 (two rounds)
//           33 + 9; 64 requests of 16 heads 37 + 4, 27 + 4, 34 + 5
//           More than 128 blocks stay whole.  129 to 255 of them leave compute
//           units idle, and the others run faster for it (132 blocks of 32 fp8
//           tiles 70 us, 252 of them 74): requests of 128 heads over 2048 rows
//           whole | in halves | in thirds
//             33   70 | 79 + 8  | 60 + 9       40   70 | 79 + 9 | 62 + 10
//             48   71 | 81 + 11 | 89 + 12      63   74 | 83 + 14
//             65  138 | 118 + 14 | 118 + 15    96  141 | 124 + 19 | 153 + 21
//           over 512 rows 33: 26 | - | 34 + 9, 65: 50 | 54 + 14; 129 requests
//           of 16 heads 70 | - | 63 + 6
AttendPlan attend_plan(int32_t n, int32_t nq, int32_t heads, int32_t d_v, int32_t rows, bool mapped)
{
    AttendPlan p{};
    const int64_t units = mapped ? (int64_t)n * nq : n;
    const int32_t unit_rows = mapped ? heads : nq * heads;
    p.block = unit_rows <= 16 ? 16 : kMaxBlock;
    p.groups = (unit_rows + p.block - 1) / p.block;
    const int64_t tiles = (rows + kTile - 1) / kTile;
    int64_t shares = kWorkgroups / (units * p.groups);
    shares = shares < tiles ? shares : tiles;
    p.shares = (int32_t)(shares < 1 ? 1 : shares);
    p.workspace = p.shares > 1 ? partial_bytes(units * p.shares * unit_rows, d_v) : 0;
    return p;
}

// Over all smaller calls: their query rows times shares are at most the query
// rows times tiles, and at most a block for each workgroup.
int64_t attend_workspace_bound(int32_t n, int32_t nq, int32_t heads, int32_t d_v, int32_t rows)
{
    const int64_t all = (int64_t)n * nq * heads, tiles = (rows + kTile - 1) / kTile;
    const int64_t most = all * tiles;
    if (tiles < 2)
        return 0;
    return partial_bytes(most < kWorkgroups * kMaxBlock ? most : kWorkgroups * kMaxBlock, d_v);
}

hipError_t launch_attend(const kvr_ctx *c, const kvr_attend_call &call, const AttendPlan &plan,
                         hipStream_t s)
{
    AttendArgs a{};
    a.sh = c->shape;
    a.layers = c->layers_d;
    a.c = call;
    if (call.rows)
        a.c.layer = 0;  // (not checked then, and not used)
    a.units = call.map ? call.n * call.nq : call.n;
    a.unit_rows = call.map ? call.heads : call.nq * call.heads;
    a.groups = plan.groups;
    a.shares = plan.shares;
    a.wide = reinterpret_cast<uintptr_t>(call.q) % 16 == 0 && call.q_stride_entry % 8 == 0 &&
             call.q_stride_query % 8 == 0 && call.q_stride_head % 8 == 0;
    const int64_t parts = (int64_t)a.units * a.shares;
    a.partial = static_cast<float *>(call.workspace);
    a.stat = a.partial ? a.partial + parts * a.unit_rows * call.d_v : nullptr;
    const dim3 grid((unsigned)((parts * a.groups + 7) / 8 * 8));
    hipError_t e = call.format == KVR_ROW_FP8    ? launch_format<KVR_ROW_FP8>(c, a, plan.block, grid, s)
                   : call.format == KVR_ROW_BF16 ? launch_format<KVR_ROW_BF16>(c, a, plan.block, grid, s)
                                                 : launch_format<KVR_ROW_F16>(c, a, plan.block, grid, s);
    if (e != hipSuccess || a.shares == 1)
        return e;
    if (call.format == KVR_ROW_F16)
        return call.d_v == 512 ? launch_join<_Float16, 512>(c, a, s)
                               : launch_join<_Float16, 256>(c, a, s);
    return call.d_v == 512 ? launch_join<__bf16, 512>(c, a, s) : launch_join<__bf16, 256>(c, a, s);
}

}  // namespace kvr
