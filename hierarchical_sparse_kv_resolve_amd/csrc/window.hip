// The drafter's window in 8 bits ("Adaptive DHiSparse: Speculative Decoding over
// a Load-Adaptive KV Hierarchy", section "How it works", paragraph "Speculative
// state": the drafter stores just the rows it can still see): new tokens' keys
// and values into the ring's blocks, the visible rows back, and the lengths.
// window_attend.hip reads the same blocks.
//
// A block holds 64 tokens of one head: keys [64][d], values [d][64], so that
// the matrix instructions of the attention take both straight from memory.
// Its scales are powers of two, 2^e with the smallest e >= -100 for which
// max|x| <= 448 * 2^e: a code that moves to another scale keeps its bits unless
// it falls below the smallest normal code, scaling in the attention is exact in
// bf16, and no division is needed.
//
// Writing: one workgroup for each touched block and head.  It reads the block's
// codes if rows of it are kept, finds what is not finite, the maxima and the
// scales, then writes the block.  Values turn through LDS (codes of [token][d] to
// [d][token]).  A block and head is the unit because its scale depends on all of it:
// nothing is exchanged between workgroups.
//
// What they take (one MI355X, 8 heads of 128, bf16, other tokens in each call and the
// lengths advanced after it): 8 chunks of 4096 tokens 45 to 47 us, 201 MB read and
// written at 4.3 to 4.5 TB/s; one token of 64 requests 8.1 us, of one 6.4, latency:
// lengths, then codes and new values, then three exchanges through LDS.  (Pieces
// compared with what they replace and written where they differ: 50, 8.1 and 6.8 us.)
// 32 windows of 4096 rows read back 165 us, 805 MB at 4.9 TB/s, the rate of a large
// copy; one of 1024 rows 5.0 us.
#include "block.h"
#include "draft.h"
#include "kvr_internal.h"
#include "rowformat.h"
#include "values.h"

namespace kvr {
namespace {

constexpr int NT = 256;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct WriteArgs {
    Window w;
    kvr_draft_write_call c;
    int32_t blocks;  // touched blocks of an entry, at most
    bool wide;
};

constexpr uint32_t kInfBits = 0x7F800000u;
// 248 * 2^120: from here on the nearest code of a block's largest scale is 256, which
// would stand for 2^128.
constexpr uint32_t kPastBits = 0x7F780000u;

// 16 consecutive values.
template <typename T>
struct Run {
    static constexpr int kPer = 16 / sizeof(T);  // values of 16 bytes
    typedef T vec __attribute__((ext_vector_type(kPer)));
    vec v[16 / kPer];

    __device__ __forceinline__ float at(int i) const { return (float)v[i / kPer][i % kPer]; }
    __device__ __forceinline__ void set(int i, float x) { v[i / kPer][i % kPer] = (T)x; }
    __device__ __forceinline__ void load(const T *p, bool wide)
    {
        if (wide) {
#pragma unroll
            for (int i = 0; i < 16 / kPer; ++i)
                v[i] = *reinterpret_cast<const vec *>(p + i * kPer);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i / kPer][i % kPer] = p[i];
        }
    }
};

// The largest magnitude, as the bits of a float.
template <typename T>
__device__ __forceinline__ uint32_t largest(const Run<T> &x)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(x.at(i)) & 0x7FFFFFFFu;
        top = top > u ? top : u;
    }
    return top;
}

// Values as codes can hold them: 240 * 2^120 for those past it, 0 for what is no number.
template <typename T>
__device__ __forceinline__ void hold(Run<T> &x)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = x.at(i), size = fabsf(y);
        x.set(i, size < __uint_as_float(kPastBits) ? y
                 : size < __builtin_inff()         ? copysignf(240.f * 0x1p120f, y)
                                                   : 0.f);
    }
}

// The smallest e, as a scale byte, with top <= 448 * 2^e, top's bits being u.
__device__ __forceinline__ int scale_for(uint32_t u)
{
    // 448 = 1.75 * 2^8
    const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u);
    return e > kMinScale ? e : kMinScale;
}

// What codes of scale byte `from` are multiplied by to have scale byte `to`.  A
// code other than 0 has at least 2^-9 of its scale and at most 2^9 of the new one,
// so only blocks of zeros go beyond 2^18 (held to 2^32: no infinity).
__device__ __forceinline__ float move_between(int from, int to)
{
    const int e = kBias + from - to;
    return scale_value(e < 1 ? 1 : e > kBias + 32 ? kBias + 32 : e);
}

__device__ __forceinline__ void widen16(const u32x4 &codes, float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[i], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[i], true);
        x[4 * i] = a[0], x[4 * i + 1] = a[1], x[4 * i + 2] = b[0], x[4 * i + 3] = b[1];
    }
}

// The codes of 16 values times `inv`.
__device__ __forceinline__ u32x4 narrow16(const float (&x)[16], float inv)
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pack_e4m3(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
    return v;
}

template <typename T>
__device__ __forceinline__ u32x4 narrow(const Run<T> &x, float inv)
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pack_e4m3(x.at(4 * i) * inv, x.at(4 * i + 1) * inv, x.at(4 * i + 2) * inv,
                         x.at(4 * i + 3) * inv);
    return v;
}

// Codes of 16 tokens, all but those of `keep` set to 0.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 v, uint32_t keep)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m |= (keep >> (4 * i + j)) & 1 ? 0xFFu << (8 * j) : 0u;
        v[i] &= m;
    }
    return v;
}

template <int D, typename T>
__global__ __launch_bounds__(NT) void write_kernel(WriteArgs a)
{
    constexpr int kPieces = kBlock * D / 16 / NT;  // 16-byte pieces of a thread, keys or values
    constexpr int kRow = D / 16;                   // pieces of a token
    __shared__ uint32_t sBad[2];                   // tokens that are not finite
    __shared__ uint32_t sTop[2];                   // maxima, as bits
    __shared__ __attribute__((aligned(16))) uint8_t sV[kBlock][D + 16];

    const int h = blockIdx.y, tid = threadIdx.x;
    const int i = blockIdx.x / a.blocks, t = blockIdx.x % a.blocks;
    const Entry e = entry_of(a.w, a.c.req_ids, a.c.count, a.c.rows, i);
    if (a.c.status && h == 0 && t == 0 && tid == 0)
        a.c.status[i] = e.status;
    if (e.status != KVR_OK || e.count == 0)
        return;
    const int64_t first = (e.length / kBlock + (int64_t)t) * kBlock;  // position of slot 0
    if (first >= (int64_t)e.length + e.count)
        return;
    const int64_t unit =
        ((int64_t)e.r * a.w.blocks + (int)(first / kBlock % a.w.blocks)) * a.w.kv_heads + h;
    uint8_t *codes = a.w.codes + unit * (2 * kBlock * D);
    uint8_t *scales = a.w.scales + unit * 2;

    // which tokens are new, and which slots hold rows that are kept: what a slot holds is
    // the last position below `high` that falls to it (a dropped token may have taken the
    // place of a row of this lap that is below `length`)
    const int64_t pos = first + lane_id();
    const bool is_new = pos >= e.length && pos < (int64_t)e.length + e.count;
    const int64_t was = pos < e.high ? pos : pos - a.w.C;
    const uint64_t fresh = __ballot(is_new);
    const uint64_t live = __ballot(!is_new && was >= 0 && was < e.length &&
                                   was >= (int64_t)e.high - a.w.C);
    if (tid < 2) {
        sBad[tid] = 0;
        sTop[tid] = 0;
    }

    // old codes, and the new values: piece p of a thread is q = p * NT + tid;
    // keys (and values as they come): token q / kRow, values of d q % kRow * 16
    u32x4 ok[kPieces], ov[kPieces];
    int old_k = 0, old_v = 0;
    if (live) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            ok[p] = *reinterpret_cast<const u32x4 *>(codes + (p * NT + tid) * 16);
            ov[p] = *reinterpret_cast<const u32x4 *>(codes + kBlock * D + (p * NT + tid) * 16);
        }
        old_k = scales[0];
        old_v = scales[1];
    }
    Run<T> nk[kPieces], nv[kPieces];  // (kept in their type: half the registers)
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int q = p * NT + tid, tok = q / kRow, d = q % kRow * 16;
        if ((fresh >> tok) & 1) {
            const int64_t j = first + tok - e.length;
            nk[p].load(static_cast<const T *>(a.c.k) + i * a.c.k_stride_entry +
                           j * a.c.k_stride_token + h * a.c.k_stride_head + d, a.wide);
            nv[p].load(static_cast<const T *>(a.c.v) + i * a.c.v_stride_entry +
                           j * a.c.v_stride_token + h * a.c.v_stride_head + d, a.wide);
        }
    }
    __syncthreads();
    // maxima as bits, in which an infinity or a NaN is above all
    uint32_t top_k = 0, top_v = 0, piece_k[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int tok = (p * NT + tid) / kRow;
        piece_k[p] = 0;
        if ((fresh >> tok) & 1) {
            piece_k[p] = largest(nk[p]);
            uint32_t piece_v = largest(nv[p]);
            const bool bad = piece_k[p] >= kInfBits || piece_v >= kInfBits;
            if (bad)
                atomicOr(&sBad[tok / 32], 1u << (tok % 32));
            if (piece_k[p] >= kPastBits) {
                hold(nk[p]);
                piece_k[p] = largest(nk[p]);
            }
            if (piece_v >= kPastBits) {
                hold(nv[p]);
                piece_v = largest(nv[p]);
            }
            top_v = top_v > piece_v ? top_v : piece_v;
        }
    }
    __syncthreads();
    const uint64_t bad = sBad[0] | (uint64_t)sBad[1] << 32;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int tok = (p * NT + tid) / kRow;
        if ((fresh & ~bad) >> tok & 1)
            top_k = top_k > piece_k[p] ? top_k : piece_k[p];
    }
    if (live) {
        float old_top_k = 0.f, old_top_v = 0.f;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int q = p * NT + tid;
            float x[16];
            if ((live >> (q / kRow)) & 1) {
                widen16(ok[p], x);
#pragma unroll
                for (int y = 0; y < 16; ++y)
                    old_top_k = fmaxf(old_top_k, fabsf(x[y]));  // (a NaN is no maximum)
            }
            widen16(keep_bytes(ov[p], (uint32_t)(live >> (q % 4 * 16))), x);
#pragma unroll
            for (int y = 0; y < 16; ++y)
                old_top_v = fmaxf(old_top_v, fabsf(x[y]));
        }
        const uint32_t k = __float_as_uint(old_top_k * scale_value(old_k));
        const uint32_t v = __float_as_uint(old_top_v * scale_value(old_v));
        top_k = top_k > k ? top_k : k;
        top_v = top_v > v ? top_v : v;
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const uint32_t k = __shfl_xor(top_k, m), v = __shfl_xor(top_v, m);
        top_k = top_k > k ? top_k : k;
        top_v = top_v > v ? top_v : v;
    }
    if (lane_id() == 0) {
        atomicMax(&sTop[0], top_k);
        atomicMax(&sTop[1], top_v);
    }
    __syncthreads();
    const int e_k = scale_for(sTop[0]), e_v = scale_for(sTop[1]);
    // 2^-e; e is in [-100, 120]
    const float inv_k = scale_value(2 * kBias - e_k), inv_v = scale_value(2 * kBias - e_v);
    const float move_k = move_between(old_k, e_k), move_v = move_between(old_v, e_v);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int q = p * NT + tid, tok = q / kRow, d = q % kRow * 16;
        u32x4 v = {};
        if ((fresh >> tok) & 1) {
            v = (bad >> tok) & 1 ? u32x4{0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu}
                                 : narrow(nk[p], inv_k);
            *reinterpret_cast<u32x4 *>(&sV[tok][d]) = narrow(nv[p], inv_v);
        } else if ((live >> tok) & 1) {
            v = ok[p];
            if (e_k != old_k) {
                float x[16];
                widen16(v, x);
                v = narrow16(x, move_k);
            }
        }
        *reinterpret_cast<u32x4 *>(codes + q * 16) = v;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int q = p * NT + tid, d = q / 4, t0 = q % 4 * 16;
        u32x4 v = {};
        if (live) {
            v = keep_bytes(ov[p], (uint32_t)(live >> t0));
            if (e_v != old_v) {
                float x[16];
                widen16(v, x);
                v = narrow16(x, move_v);
            }
        }
        const uint32_t take = (uint32_t)(fresh >> t0) & 0xFFFFu;
#pragma unroll
        for (int y = 0; y < 16; ++y)
            if ((take >> y) & 1)
                v[y / 4] |= (uint32_t)sV[t0 + y][d] << (y % 4 * 8);
        *reinterpret_cast<u32x4 *>(codes + kBlock * D + q * 16) = v;
    }
    if (tid == 0) {
        scales[0] = (uint8_t)e_k;
        scales[1] = (uint8_t)e_v;
    }
}

struct ReadArgs {
    Window w;
    const int32_t *req_ids;
    void *k, *v;
    int32_t *visible, *status;
    int32_t blocks;  // blocks that a window can touch
};

// One workgroup for each block of an entry's window and head.
template <int D, typename T>
__global__ __launch_bounds__(NT) void read_kernel(ReadArgs a)
{
    constexpr int kPieces = kBlock * D / 16 / NT;
    constexpr int kRow = D / 16;
    __shared__ __attribute__((aligned(16))) uint8_t sV[D][kBlock + 4];
    const int h = blockIdx.y, tid = threadIdx.x;
    const int i = blockIdx.x / a.blocks, t = blockIdx.x % a.blocks;
    Entry e = entry_of(a.w, a.req_ids, nullptr, 0, i);
    const int32_t lo = e.length > a.w.W ? e.length - a.w.W : 0;
    if (e.status == KVR_OK && lo < e.high - a.w.C)
        e.status = KVR_E_RANGE;
    if (h == 0 && t == 0 && tid == 0) {
        if (a.status)
            a.status[i] = e.status;
        if (a.visible && e.status == KVR_OK)
            a.visible[i] = e.length - lo;
    }
    if (e.status != KVR_OK)
        return;
    const int64_t first = (lo / kBlock + (int64_t)t) * kBlock;
    if (first >= e.length)
        return;
    const int64_t unit =
        ((int64_t)e.r * a.w.blocks + (int)(first / kBlock % a.w.blocks)) * a.w.kv_heads + h;
    const uint8_t *codes = a.w.codes + unit * (2 * kBlock * D);
    const float k_unit = scale_value(a.w.scales[unit * 2]);
    const float v_unit = scale_value(a.w.scales[unit * 2 + 1]);
    u32x4 kc[kPieces], vc[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        kc[p] = *reinterpret_cast<const u32x4 *>(codes + (p * NT + tid) * 16);
        vc[p] = *reinterpret_cast<const u32x4 *>(codes + kBlock * D + (p * NT + tid) * 16);
    }
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int q = p * NT + tid;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            *reinterpret_cast<uint32_t *>(&sV[q / 4][q % 4 * 16 + 4 * y]) = vc[p][y];
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int q = p * NT + tid, tok = q / kRow, d = q % kRow * 16;
        const int64_t pos = first + tok;
        if (pos < lo || pos >= e.length)
            continue;
        const int64_t at = (((int64_t)i * a.w.W + (pos - lo)) * a.w.kv_heads + h) * D + d;
        float x[16];
        widen16(kc[p], x);
#pragma unroll
        for (int y = 0; y < 16; ++y)
            x[y] *= k_unit;
        store_run<16>(static_cast<T *>(a.k) + at, true, x);
        u32x4 v;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            v[y] = sV[d + 4 * y][tok] | (uint32_t)sV[d + 4 * y + 1][tok] << 8 |
                   (uint32_t)sV[d + 4 * y + 2][tok] << 16 | (uint32_t)sV[d + 4 * y + 3][tok] << 24;
        widen16(v, x);
#pragma unroll
        for (int y = 0; y < 16; ++y)
            x[y] *= v_unit;
        store_run<16>(static_cast<T *>(a.v) + at, true, x);
    }
}

__global__ void advance_kernel(Window w, int32_t n, const int32_t *req_ids, int32_t rows,
                               const int32_t *count, int32_t *length, int32_t *high,
                               int32_t *status)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n)
        return;
    const Entry e = entry_of(w, req_ids, count, rows, i);
    if (status)
        status[i] = e.status;
    if (e.status != KVR_OK)
        return;
    length[e.r] = e.length + e.count;
    if (e.length + e.count > e.high)
        high[e.r] = e.length + e.count;
}

template <int D>
hipError_t launch_write_dim(const WriteArgs &a, dim3 grid, hipStream_t s)
{
    if (a.c.value_type == KVR_VALUE_F32)
        return launch(nullptr, 0, write_kernel<D, float>, grid, dim3(NT), 0, s, a);
    if (a.c.value_type == KVR_VALUE_BF16)
        return launch(nullptr, 0, write_kernel<D, __bf16>, grid, dim3(NT), 0, s, a);
    return launch(nullptr, 0, write_kernel<D, _Float16>, grid, dim3(NT), 0, s, a);
}

template <int D>
hipError_t launch_read_dim(const ReadArgs &a, int32_t value_type, dim3 grid, hipStream_t s)
{
    if (value_type == KVR_VALUE_F32)
        return launch(nullptr, 0, read_kernel<D, float>, grid, dim3(NT), 0, s, a);
    if (value_type == KVR_VALUE_BF16)
        return launch(nullptr, 0, read_kernel<D, __bf16>, grid, dim3(NT), 0, s, a);
    return launch(nullptr, 0, read_kernel<D, _Float16>, grid, dim3(NT), 0, s, a);
}

}  // namespace

hipError_t launch_draft_write(const kvr_draft *d, const kvr_draft_write_call &c, hipStream_t s)
{
    WriteArgs a{};
    a.w = window_of(d, c.layer);
    a.c = c;
    a.blocks = (c.rows + kBlock - 2) / kBlock + 1;
    const int64_t e = 16 / value_bytes(c.value_type);
    a.wide = (reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) % 16 == 0 &&
             (c.k_stride_entry | c.k_stride_token | c.k_stride_head | c.v_stride_entry |
              c.v_stride_token | c.v_stride_head) % e == 0;
    const dim3 grid((unsigned)((int64_t)c.n * a.blocks), (unsigned)d->kv_heads);
    return d->d_head == 64    ? launch_write_dim<64>(a, grid, s)
           : d->d_head == 128 ? launch_write_dim<128>(a, grid, s)
                              : launch_write_dim<256>(a, grid, s);
}

hipError_t launch_draft_read(const kvr_draft *d, int32_t layer, int32_t n, const int32_t *req_ids,
                             int32_t value_type, void *k, void *v, int32_t *visible,
                             int32_t *status, hipStream_t s)
{
    ReadArgs a{};
    a.w = window_of(d, layer);
    a.req_ids = req_ids;
    a.k = k;
    a.v = v;
    a.visible = visible;
    a.status = status;
    a.blocks = (d->W + kBlock - 2) / kBlock + 1;
    const dim3 grid((unsigned)((int64_t)n * a.blocks), (unsigned)d->kv_heads);
    return d->d_head == 64    ? launch_read_dim<64>(a, value_type, grid, s)
           : d->d_head == 128 ? launch_read_dim<128>(a, value_type, grid, s)
                              : launch_read_dim<256>(a, value_type, grid, s);
}

hipError_t launch_draft_advance(const kvr_draft *d, int32_t n, const int32_t *req_ids,
                                int32_t rows, const int32_t *count, int32_t *status,
                                hipStream_t s)
{
    Window w{};
    w.n_req = d->n_req;
    w.length = d->length;
    w.high = d->high;
    return launch(nullptr, 0, advance_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, w,
                  n, req_ids, rows, count, d->length, d->high, status);
}

int check_draft_stream(const kvr_draft *d, int32_t n, hipStream_t s)
{
    if (int rc = draft_prologue(d, n, s))
        return rc;
    if (s) {
        hipDevice_t dev = -1;
        const hipError_t e = hipStreamGetDevice(s, &dev);
        if (e != hipSuccess)
            return api_fail(KVR_E_HIP, "hipStreamGetDevice: %s", hipGetErrorString(e));
        if (dev != d->device)
            return api_fail(KVR_E_ARG, "the stream is on device %d, not the ring's device %d",
                            (int)dev, d->device);
    }
    return KVR_OK;
}

int check_draft_kv(const kvr_draft *d, int32_t layer, int32_t n, hipStream_t s)
{
    if (int rc = check_draft_stream(d, n, s))
        return rc;
    if (!d->codes)
        return api_fail(KVR_E_ARG, "no K/V layers bound");
    if (layer < 0 || layer >= d->kv_layers)
        return api_fail(KVR_E_ARG, "layer %d outside [0, %d)", layer, d->kv_layers);
    return KVR_OK;
}

namespace {

int launched(hipError_t e, const char *what)
{
    if (e != hipSuccess)
        return api_fail(KVR_E_HIP, "%s: %s", what, hipGetErrorString(e));
    return api_ok();
}

}  // namespace
}  // namespace kvr

extern "C" {

int kvr_draft_bind_kv(kvr_draft *d, int32_t n_layers, int32_t kv_heads, int32_t d_head,
                      void *codes, uint8_t *scales)
{
    if (!d)
        return kvr::api_fail(KVR_E_ARG, "null drafter ring");
    if (d->C % kvr::kBlock != 0)
        return kvr::api_fail(KVR_E_ARG, "the ring's capacity %d is not a multiple of %d", d->C,
                             kvr::kBlock);
    if (n_layers < 1 || kv_heads < 1 || kv_heads > 256 ||
        (d_head != 64 && d_head != 128 && d_head != 256))
        return kvr::api_fail(KVR_E_ARG, "n_layers must be >= 1, kv_heads in [1, 256], d_head 64, "
                                        "128 or 256");
    if (!codes || !scales || reinterpret_cast<uintptr_t>(codes) % 16 != 0)
        return kvr::api_fail(KVR_E_ARG, "codes (aligned to 16 bytes) and scales are required");
    d->kv_layers = n_layers;
    d->kv_heads = kv_heads;
    d->d_head = d_head;
    d->codes = static_cast<uint8_t *>(codes);
    d->scales = scales;
    return kvr::api_ok();
}

int kvr_draft_write_kv(kvr_draft *d, const kvr_draft_write_call *call, void *stream)
{
    if (!d)
        return kvr::api_fail(KVR_E_ARG, "null drafter ring");
    if (!call)
        return kvr::api_fail(KVR_E_ARG, "null call");
    const kvr_draft_write_call &c = *call;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (int rc = kvr::check_draft_kv(d, c.layer, c.n, s))
        return rc;
    if (!kvr::value_type_ok(c.value_type))
        return kvr::api_fail(KVR_E_ARG, "unknown value type %d", c.value_type);
    if (c.rows < 0 || c.rows > d->C - (kvr::kBlock - 1))
        return kvr::api_fail(KVR_E_ARG, "rows must be in [0, capacity - %d]", kvr::kBlock - 1);
    if (c.k_stride_entry < 0 || c.k_stride_token < 0 || c.k_stride_head < 0 ||
        c.v_stride_entry < 0 || c.v_stride_token < 0 || c.v_stride_head < 0)
        return kvr::api_fail(KVR_E_ARG, "negative stride");
    if (c.n > 0 && c.rows > 0 && (!c.k || !c.v))
        return kvr::api_fail(KVR_E_ARG, "k and v are required");
    const uintptr_t e = (uintptr_t)kvr::value_bytes(c.value_type);
    if (reinterpret_cast<uintptr_t>(c.k) % e != 0 || reinterpret_cast<uintptr_t>(c.v) % e != 0)
        return kvr::api_fail(KVR_E_ARG, "k or v is not aligned");
    if ((int64_t)c.n * ((c.rows + kvr::kBlock - 2) / kvr::kBlock + 1) >= (1 << 24))
        return kvr::api_fail(KVR_E_ARG, "too many blocks in one call");
    if (c.n == 0)
        return kvr::api_ok();
    return kvr::launched(kvr::launch_draft_write(d, c, s), "drafter K/V write launch");
}

int kvr_draft_read_kv(kvr_draft *d, int32_t layer, int32_t n, const int32_t *req_ids,
                      int32_t value_type, void *k, void *v, int32_t *visible, int32_t *status,
                      void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (int rc = kvr::check_draft_kv(d, layer, n, s))
        return rc;
    if (!kvr::value_type_ok(value_type))
        return kvr::api_fail(KVR_E_ARG, "unknown value type %d", value_type);
    if (n > 0 && (!k || !v))
        return kvr::api_fail(KVR_E_ARG, "k and v are required");
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 != 0)
        return kvr::api_fail(KVR_E_ARG, "k or v is not aligned to 16 bytes");
    if ((int64_t)n * ((d->W + kvr::kBlock - 2) / kvr::kBlock + 1) >= (1 << 24))
        return kvr::api_fail(KVR_E_ARG, "too many blocks in one call");
    if (n == 0)
        return kvr::api_ok();
    return kvr::launched(kvr::launch_draft_read(d, layer, n, req_ids, value_type, k, v, visible,
                                                status, s),
                         "drafter K/V read launch");
}

int kvr_draft_advance(kvr_draft *d, int32_t n, const int32_t *req_ids, int32_t rows,
                      const int32_t *count, int32_t *status, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (int rc = kvr::check_draft_stream(d, n, s))
        return rc;
    if (rows < 0)
        return kvr::api_fail(KVR_E_ARG, "negative row count");
    if (n == 0)
        return kvr::api_ok();
    return kvr::launched(kvr::launch_draft_advance(d, n, req_ids, rows, count, status, s),
                         "drafter advance launch");
}

int64_t kvr_draft_attend_workspace(const kvr_draft *d, int32_t n, int32_t nq, int32_t heads)
{
    if (!d || !d->codes)
        return kvr::api_fail(KVR_E_ARG, "no K/V layers bound");
    if (n < 0 || nq < 1 || heads < 1 || heads > 4096 || heads % d->kv_heads != 0 ||
        (int64_t)n * nq * heads > (1 << 22))
        return kvr::api_fail(KVR_E_ARG, "n must be >= 0, nq >= 1, heads a multiple of the K/V "
                                        "heads up to 4096, n * nq * heads at most 2^22");
    kvr::api_ok();
    return kvr::draft_workspace_bound(n, nq, heads, d->kv_heads, d->d_head, d->W);
}

int kvr_draft_attend(kvr_draft *d, const kvr_draft_attend_call *call, void *stream)
{
    if (!d)
        return kvr::api_fail(KVR_E_ARG, "null drafter ring");
    if (!call)
        return kvr::api_fail(KVR_E_ARG, "null call");
    const kvr_draft_attend_call &c = *call;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (int rc = kvr::check_draft_kv(d, c.layer, c.n, s))
        return rc;
    if (c.mask != KVR_DRAFT_CAUSAL && c.mask != KVR_DRAFT_WHOLE && c.mask != KVR_DRAFT_KEPT)
        return kvr::api_fail(KVR_E_ARG, "unknown mask %d", c.mask);
    if (c.nq < 1 || c.heads < 1 || c.heads > 4096 || c.heads % d->kv_heads != 0 ||
        (int64_t)c.n * c.nq * c.heads > (1 << 22))
        return kvr::api_fail(KVR_E_ARG, "nq must be >= 1, heads a multiple of the K/V heads up to "
                                        "4096, n * nq * heads at most 2^22");
    if (!(fabsf(c.scale) < 0x1p127f))
        return kvr::api_fail(KVR_E_ARG, "scale must be finite and below 2^127");
    if (c.mask == KVR_DRAFT_CAUSAL && c.nq > d->C - d->W + 1)
        return kvr::api_fail(KVR_E_ARG, "%d causal queries: the ring keeps the rows of %d", c.nq,
                             d->C - d->W + 1);
    if (c.mask == KVR_DRAFT_WHOLE && c.nq > d->C)
        return kvr::api_fail(KVR_E_ARG, "%d new tokens in a ring of %d", c.nq, d->C);
    if (c.n > 0 && (!c.q || !c.out))
        return kvr::api_fail(KVR_E_ARG, "q and out are required");
    if (c.q_stride_entry < 0 || c.q_stride_query < 0 || c.q_stride_head < 0)
        return kvr::api_fail(KVR_E_ARG, "negative stride of q");
    if (reinterpret_cast<uintptr_t>(c.q) % 2 != 0 || reinterpret_cast<uintptr_t>(c.out) % 16 != 0)
        return kvr::api_fail(KVR_E_ARG, "q or out is not aligned");
    if (c.n == 0)
        return kvr::api_ok();
    const int64_t tokens = (int64_t)d->W + (c.mask == KVR_DRAFT_CAUSAL ? c.nq - 1 : 0);
    const kvr::DraftPlan plan =
        kvr::draft_plan(c.n, c.nq, c.heads, d->kv_heads, d->d_head, (int32_t)tokens);
    if (plan.workspace > 0) {
        if (!c.workspace || c.workspace_bytes < (size_t)plan.workspace)
            return kvr::api_fail(KVR_E_ARG, "the workspace has %zu bytes, the call needs %lld",
                                 c.workspace ? c.workspace_bytes : 0, (long long)plan.workspace);
        if (reinterpret_cast<uintptr_t>(c.workspace) % 16 != 0)
            return kvr::api_fail(KVR_E_ARG, "the workspace is not aligned to 16 bytes");
    }
    return kvr::launched(kvr::launch_draft_attend(d, c, plan, s), "drafter attention launch");
}

}  // extern "C"
