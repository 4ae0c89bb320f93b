// Attention of new tokens' queries over the drafter's window in 8 bits
// ("Adaptive DHiSparse: Speculative Decoding over a Load-Adaptive KV Hierarchy",
// section "How it works", paragraph "Speculative state").
//
// For a query row x (a head of a query) over the tokens j that it sees:
//   t_j = log2(e) * scale * (q . key_j),  p_j = 2^(t_j - m),  l = sum p_j,
//   out = sum p_j value_j / l,            lse = ln 2 * (m + log2 l)
// with one pass over the tokens: m is a reference at most 8 below the running
// maximum; when a score exceeds it by more, the maximum becomes the reference
// and l and the sums are scaled down.
//
// A wave owns MB blocks of 16 query rows of one K/V head and walks ring blocks
// of 64 tokens, 16-byte loads straight from memory into the operands of
// 16x16x32 MFMA, the next block's on their way beside the products:
//   scores  (keys x queries) 4 tiles of 16 tokens.  Row 4 g + k of tile j is
//           token 16 g + 4 j + k, so that lane group g ends up with the
//           probabilities of tokens 16 g .. 16 g + 15,
//   values  which are, 8 at a time, the other operand's columns: the values lie
//           [d][64 tokens], and a lane reads the same 16 tokens of a dimension.
// Nothing passes through LDS and no wave waits for another; a query row stays in
// one lane (mod 16), so maxima and sums are the lane's own but for one exchange
// between lane groups where a reference changes, and one at the end.
//
// Codes become bf16 exactly, with their block's scale (a power of two): the
// keys' is folded into log2(e) * scale, the values' into the conversion.
#include "block.h"
#include "draft.h"
#include "kvr_internal.h"

namespace kvr {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 frag __attribute__((ext_vector_type(8)));

constexpr float kSlack = 8.f;  // p is at most 2^8

struct AttendArgs {
    Window w;
    kvr_draft_attend_call c;
    int32_t group;   // query heads of a K/V head
    int32_t tiles;   // workgroups that the query rows of an entry and head take
    int32_t shares;
    uint32_t jobs;
    bool wide;       // q may be read 16 bytes at a time
    float *partial;  // [n][kv_heads][shares][nq * group][d], with shares > 1
    float *stat;     // [n][kv_heads][shares][nq * group][2]: m, l
};

__device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 8 e4m3 codes times a power of two as bf16 values.
__device__ __forceinline__ frag widen(uint32_t lo, uint32_t hi, float unit)
{
    frag f;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, unit, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, unit, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, unit, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, unit, true);
    f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1];
    f[4] = c[0], f[5] = c[1], f[6] = d[0], f[7] = d[1];
    return f;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Position after the last one that query j sees.
__device__ __forceinline__ int end_of(int mask, const Entry &e, int j)
{
    return mask == KVR_DRAFT_CAUSAL ? e.length + j + 1
           : mask == KVR_DRAFT_WHOLE ? e.length + e.count
                                     : e.length;
}

// The entry with what the call's mask asks of the ring.
__device__ __forceinline__ Entry attend_entry(const AttendArgs &a, int i)
{
    Entry e = entry_of(a.w, a.c.req_ids, a.c.count, a.c.nq, i);
    if (e.status == KVR_OK && e.count > 0) {
        // positions written: before the call's tokens, or with them
        const int32_t top =
            a.c.mask != KVR_DRAFT_KEPT && e.length + e.count > e.high ? e.length + e.count : e.high;
        const int32_t end = end_of(a.c.mask, e, 0);
        const int32_t lo = end > a.w.W ? end - a.w.W : 0;
        if (lo < top - a.w.C)
            e.status = KVR_E_RANGE;
    }
    return e;
}

template <int D, int MB, int NW, bool SPLIT>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
void attend_kernel(AttendArgs a)
{
    constexpr int kRows = 16 * MB;          // query rows of a wave
    constexpr int kSteps = D / 32;          // MFMA steps of a score
    constexpr int kLoads = D / 64;          // 16-byte loads of a key in a lane
    constexpr int kCols = D / 16;           // blocks of 16 value columns
    __shared__ __attribute__((aligned(16))) float sO[SPLIT ? NW * kRows * (D + 4) : 1];
    __shared__ float sStat[SPLIT ? NW * kRows * 2 : 1];

    const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());

    // Workgroups are dealt to the 8 XCDs in turn: each XCD takes a run of
    // neighbours, so that its L2 serves the tokens of one head to all of them.
    const uint32_t job = (blockIdx.x & 7) * ((a.jobs + 7) / 8) + blockIdx.x / 8;
    if (job >= a.jobs)
        return;
    const int share = (int)(job % (uint32_t)a.shares);
    const uint32_t rest = job / (uint32_t)a.shares;
    const int tile = (int)(rest % (uint32_t)a.tiles);
    const uint32_t unit = rest / (uint32_t)a.tiles;  // entry and K/V head
    const int i = (int)(unit / (uint32_t)a.w.kv_heads), kvh = (int)(unit % (uint32_t)a.w.kv_heads);

    const Entry e = attend_entry(a, i);
    if (a.c.status && kvh == 0 && tile == 0 && share == 0 && threadIdx.x == 0)
        a.c.status[i] = e.status;
    const int x0 = SPLIT ? tile * kRows : (tile * NW + wave) * kRows;
    const int rows = e.count * a.group;  // of the entry and head
    if (e.status != KVR_OK || x0 >= rows)
        return;  // (with SPLIT, the whole workgroup)

    // blocks of tokens that the wave's rows see, and which of them all rows see whole
    const int j0 = x0 / a.group;
    const int j1 = (x0 + kRows < rows ? x0 + kRows - 1 : rows - 1) / a.group;
    const int end0 = end_of(a.c.mask, e, j0), end1 = end_of(a.c.mask, e, j1);
    const int lo0 = end0 > a.w.W ? end0 - a.w.W : 0, lo1 = end1 > a.w.W ? end1 - a.w.W : 0;
    const int b_first = lo0 / kBlock, b_last = (end1 + kBlock - 1) / kBlock;
    const int per = (b_last - b_first + a.shares - 1) / a.shares;
    const int b0 = b_first + share * per;
    const int b1 = b0 + per < b_last ? b0 + per : b_last;
    const int full0 = (lo1 + kBlock - 1) / kBlock, full1 = end0 / kBlock;

    // queries; past the last row: that row's, whose results are not written
    int hi[MB], lo[MB];  // tokens that the lane's row of each block sees
    frag qf[MB][kSteps];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int x = x0 + mb * 16 + col, xc = x < rows ? x : rows - 1;
        const int j = xc / a.group, h = kvh * a.group + xc % a.group;
        hi[mb] = end_of(a.c.mask, e, j);
        lo[mb] = hi[mb] > a.w.W ? hi[mb] - a.w.W : 0;
        const __bf16 *q = static_cast<const __bf16 *>(a.c.q) + i * a.c.q_stride_entry +
                          j * a.c.q_stride_query + h * a.c.q_stride_head;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const __bf16 *p = q + s / 2 * 64 + grp * 16 + (s & 1) * 8;
            if (a.wide) {
                qf[mb][s] = *reinterpret_cast<const frag *>(p);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    qf[mb][s][k] = p[k];
            }
            // a negative scale goes into the queries, so that the largest product
            // is the largest score
            if (a.c.scale < 0.f)
                qf[mb][s] = -qf[mb][s];
        }
    }

    float m[MB], l[MB];
    f32x4 o[kCols][MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        m[mb] = -__builtin_inff();
        l[mb] = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            o[c][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // A block's keys and values.  The next keys are loaded once the scores are
    // taken, the next values after the products, into the same registers.
    u32x4 k[4][kLoads], v[kCols];
    uint32_t k_scale = 0, v_scale = 0;
    const int64_t head_bytes = 2 * kBlock * D;
    const int64_t first = (int64_t)e.r * a.w.blocks * a.w.kv_heads + kvh;
    const int k_at = ((col >> 2) * 16 + (col & 3)) * D + grp * 16;
    const int v_at = kBlock * D + col * kBlock + grp * 16;
    auto at_block = [&](int b) { return first + (int64_t)(b % a.w.blocks) * a.w.kv_heads; };
    auto load_keys = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t *p = a.w.codes + at * head_bytes + k_at;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
                k[j][n] = *reinterpret_cast<const u32x4 *>(p + j * 4 * D + n * 64);
        k_scale = a.w.scales[at * 2];
    };
    auto load_values = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t *p = a.w.codes + at * head_bytes + v_at;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
            v[c] = *reinterpret_cast<const u32x4 *>(p + c * 16 * kBlock);
        v_scale = a.w.scales[at * 2 + 1];
    };

    // (at least the smallest normal: a scale of 0 leaves masked scores at -infinity)
    const float to_log2 = fmaxf(fabsf(a.c.scale) * 1.44269504088896340736f, 1e-37f);
    const int step = SPLIT ? NW : 1;
    int b = SPLIT ? b0 + wave : b0;
    if (b < b1) {
        load_keys(at_block(b));
        load_values(at_block(b));
    }
    for (; b < b1; b += step) {
        f32x4 s[4][MB];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                s[j][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const u32x4 w = k[j][st / 2];
                const frag kf = widen(w[(st & 1) * 2], w[(st & 1) * 2 + 1], 1.f);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                    s[j][mb] = mfma(kf, qf[mb][st], s[j][mb]);
            }
        }
        const float factor = fmaxf(to_log2 * scale_value(k_scale), 1e-37f);
        const bool more = b + step < b1;
        const int64_t at_next = at_block(b + step);
        if (more)
            load_keys(at_next);
        if (b < full0 || b >= full1) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int pos = b * kBlock + grp * 16 + j * 4 + x;
                        if (pos < lo[mb] || pos >= hi[mb])
                            s[j][mb][x] = -__builtin_inff();
                    }
        }
        frag pf[2][MB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            float top = fmaxf(fmaxf(s[0][mb][0], s[0][mb][1]), s[0][mb][2]);
#pragma unroll
            for (int x = 3; x < 15; x += 2)
                top = fmaxf(fmaxf(top, s[x / 4][mb][x % 4]), s[(x + 1) / 4][mb][(x + 1) % 4]);
            top = fmaxf(top, s[3][mb][3]) * factor;
            if (__any(top > m[mb] + kSlack)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float to = fmaxf(m[mb], top);
                const float alpha = to == -__builtin_inff() ? 1.f : exp2_hw(m[mb] - to);
                m[mb] = to;
                l[mb] *= alpha;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    o[c][mb] *= alpha;
            }
            const float ref = m[mb] == -__builtin_inff() ? 0.f : m[mb];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = exp2_hw(fmaf(s[j][mb][x], factor, -ref));
                    l[mb] += p;
                    // rounded to bf16 for the product (at most 2^-8 of it)
                    pf[j / 2][mb][(j & 1) * 4 + x] = (__bf16)p;
                }
        }
        const float v_unit = scale_value(v_scale);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const frag vf = widen(v[c][h * 2], v[c][h * 2 + 1], v_unit);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                    o[c][mb] = mfma(vf, pf[h][mb], o[c][mb]);
            }
        if (more)
            load_values(at_next);
    }

    const int64_t part = (int64_t)unit * a.shares + share;
    const int unit_rows = a.c.nq * a.group;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        l[mb] += __shfl_xor(l[mb], 16);
        l[mb] += __shfl_xor(l[mb], 32);
    }
    // row x of the head, value columns d .. d + 3 of the unnormalised sums
    auto write = [&](int x, int d, float mx, float lx, f32x4 sums) __attribute__((always_inline)) {
        if (a.shares > 1) {
            const int64_t ps = part * unit_rows + x;
            if (d == 0)
                *reinterpret_cast<float2 *>(a.stat + 2 * ps) = make_float2(mx, lx);
            *reinterpret_cast<f32x4 *>(a.partial + ps * D + d) = sums;
            return;
        }
        const int j = x / a.group, h = kvh * a.group + x % a.group;
        const int64_t at = ((int64_t)i * a.c.nq + j) * a.c.heads + h;
        const float inv = mx == -__builtin_inff() && lx == 0.f ? 0.f : 1.f / lx;
        if (d == 0 && a.c.lse)
            a.c.lse[at] = 0.69314718055994530942f * (mx + __log2f(lx));
        bf16x4 r;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            r[k] = (__bf16)(sums[k] * inv);
        *reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.c.out) + at * D + d) = r;
    };
    if constexpr (!SPLIT) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int x = x0 + mb * 16 + col;
            if (x >= rows)
                continue;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                write(x, c * 16 + grp * 4, m[mb], l[mb], o[c][mb]);
        }
    } else {
        constexpr int kStride = D + 4;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int at = wave * kRows + mb * 16 + col;
            if (grp == 0) {
                sStat[at * 2] = m[mb];
                sStat[at * 2 + 1] = l[mb];
            }
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                *reinterpret_cast<f32x4 *>(&sO[at * kStride + c * 16 + grp * 4]) = o[c][mb];
        }
        __syncthreads();
        // the waves' sums, joined in wave order
        for (int q = threadIdx.x; q < kRows * D / 4; q += NW * 64) {
            const int row = q / (D / 4), d = q % (D / 4) * 4;
            if (x0 + row >= rows)
                break;
            float mx = -__builtin_inff(), lx = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                mx = fmaxf(mx, sStat[(w * kRows + row) * 2]);
            f32x4 sums = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const int at = w * kRows + row;
                const float mw = sStat[at * 2], lw = sStat[at * 2 + 1];
                // (a wave without a score above -infinity has sums of 0 or NaN)
                const float weight = mw == -__builtin_inff() ? 1.f : exp2_hw(mw - mx);
                lx += weight * lw;
                sums += weight * *reinterpret_cast<const f32x4 *>(&sO[at * kStride + d]);
            }
            write(x0 + row, d, mx, lx, sums);
        }
    }
}

// Joins the shares of each query row: a workgroup per row, its waves taking
// every fourth share, their sums added in wave order.
constexpr int kJoinWaves = 4;
template <int D>
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(AttendArgs a)
{
    constexpr int N = D / 64;   // columns of a lane
    constexpr int kFlight = 4;  // shares in flight
    typedef float vec __attribute__((ext_vector_type(N)));
    __shared__ float sL[kJoinWaves];
    __shared__ vec sO[kJoinWaves][64];
    const int lane = lane_id(), wave = wave_id();
    const int unit_rows = a.c.nq * a.group;
    const int64_t unit = blockIdx.x / unit_rows;
    const int x = (int)(blockIdx.x % unit_rows);
    const int i = (int)(unit / a.w.kv_heads), kvh = (int)(unit % a.w.kv_heads);
    const Entry e = attend_entry(a, i);
    const int j = x / a.group, h = kvh * a.group + x % a.group;
    if (e.status != KVR_OK || j >= e.count)
        return;
    const int64_t first = unit * a.shares * unit_rows + x;
    auto stat = [&](int s) {
        return *reinterpret_cast<const float2 *>(a.stat + 2 * (first + (int64_t)s * unit_rows));
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
            w[f] = st.x == -__builtin_inff() ? 1.f : exp2_hw(st.x - m);
            ls[f] = st.y;
            part[f] = *reinterpret_cast<const vec *>(
                a.partial + (first + (int64_t)s * unit_rows) * D + lane * N);
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
    const int64_t at = ((int64_t)i * a.c.nq + j) * a.c.heads + h;
    const float inv = m == -__builtin_inff() && l == 0.f ? 0.f : 1.f / l;
    typedef __bf16 outs __attribute__((ext_vector_type(N)));
    outs v;
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = (__bf16)(o[k] * inv);
    *reinterpret_cast<outs *>(static_cast<__bf16 *>(a.c.out) + at * D + lane * N) = v;
    if (lane == 0 && a.c.lse)
        a.c.lse[at] = 0.69314718055994530942f * (m + __log2f(l));
}

constexpr int64_t kUnits = 256;  // compute units
constexpr int kWaves = 4;

// Query rows of a wave with many of them, in blocks of 16: as many as two waves
// a SIMD have registers for (one, with heads of 256).
constexpr int blocks_of_16(int d) { return d == 256 ? 1 : 2; }

int64_t partial_bytes(int64_t rows, int32_t d) { return rows * (d + 2) * (int64_t)sizeof(float); }

template <int D>
hipError_t launch_dim(const AttendArgs &a, const DraftPlan &p, dim3 grid, hipStream_t s)
{
    constexpr int MB = blocks_of_16(D);
    hipError_t e;
    if (!p.split)
        e = launch(nullptr, 0, attend_kernel<D, MB, kWaves, false>, grid, dim3(kWaves * 64), 0, s, a);
    else if (p.blocks_of_16 == 1)
        e = launch(nullptr, 0, attend_kernel<D, 1, kWaves, true>, grid, dim3(kWaves * 64), 0, s, a);
    else
        e = launch(nullptr, 0, attend_kernel<D, MB, kWaves, true>, grid, dim3(kWaves * 64), 0, s, a);
    if (e != hipSuccess || a.shares == 1)
        return e;
    const int64_t rows = (int64_t)a.c.n * a.c.nq * a.c.heads;
    return launch(nullptr, 0, join_kernel<D>, dim3((unsigned)rows), dim3(kJoinWaves * 64), 0, s, a);
}

}  // namespace

DraftPlan draft_plan(int32_t n, int32_t nq, int32_t heads, int32_t kv_heads, int32_t d_head,
                     int32_t tokens)
{
    DraftPlan p{};
    const int64_t rows = (int64_t)nq * (heads / kv_heads);  // of an entry and head
    const int64_t units = (int64_t)n * kv_heads;
    p.blocks_of_16 = rows <= 16 ? 1 : blocks_of_16(d_head);
    p.waves = kWaves;
    p.split = rows < 128;
    const int64_t tile = 16 * p.blocks_of_16 * (p.split ? 1 : kWaves);
    p.tiles = (int32_t)((rows + tile - 1) / tile);
    // a share takes a block of tokens for each wave at least
    const int64_t blocks = ((int64_t)tokens + kBlock - 1) / kBlock + 1;
    const int64_t most = (blocks + kWaves - 1) / kWaves;
    int64_t shares = 2 * kUnits / (units * p.tiles);
    shares = shares < most ? shares : most;
    p.shares = (int32_t)(shares < 1 ? 1 : shares);
    p.workspace = p.shares > 1 ? partial_bytes(units * p.shares * rows, d_head) : 0;
    return p;
}

// Over all smaller calls: their query rows times shares are at most the query
// rows times the most shares, and at most the rows of 512 workgroups.
int64_t draft_workspace_bound(int32_t n, int32_t nq, int32_t heads, int32_t kv_heads,
                              int32_t d_head, int32_t window)
{
    const int64_t blocks = ((int64_t)window + nq - 1 + kBlock - 1) / kBlock + 1;
    const int64_t most = (blocks + kWaves - 1) / kWaves;
    const int64_t all = (int64_t)n * nq * heads, tile = 32 * kWaves;
    (void)kv_heads;
    if (most < 2)
        return 0;
    return partial_bytes(all * most < 2 * kUnits * tile ? all * most : 2 * kUnits * tile, d_head);
}

hipError_t launch_draft_attend(const kvr_draft *d, const kvr_draft_attend_call &c,
                               const DraftPlan &plan, hipStream_t s)
{
    AttendArgs a{};
    a.w = window_of(d, c.layer);
    a.c = c;
    a.group = c.heads / d->kv_heads;
    a.tiles = plan.tiles;
    a.shares = plan.shares;
    a.jobs = (uint32_t)((int64_t)c.n * d->kv_heads * plan.tiles * plan.shares);
    a.wide = reinterpret_cast<uintptr_t>(c.q) % 16 == 0 &&
             (c.q_stride_entry | c.q_stride_query | c.q_stride_head) % 8 == 0;
    const int64_t parts = (int64_t)c.n * d->kv_heads * plan.shares * c.nq * a.group;
    a.partial = static_cast<float *>(c.workspace);
    a.stat = a.partial ? a.partial + parts * d->d_head : nullptr;
    const dim3 grid((a.jobs + 7) / 8 * 8);
    return d->d_head == 64    ? launch_dim<64>(a, plan, grid, s)
           : d->d_head == 128 ? launch_dim<128>(a, plan, grid, s)
                              : launch_dim<256>(a, plan, grid, s);
}

}  // namespace kvr
