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
// of 64 tokens by 16x16x32 MFMA:
//   scores  (keys x queries) 4 tiles of 16 tokens.  Row 4 g + k of tile j is
//           token 16 g + 4 j + k, so that lane group g ends up with the
//           probabilities of tokens 16 g .. 16 g + 15,
//   values  which are, 8 at a time, the other operand's columns: the values lie
//           [d][64 tokens], and a lane reads the same 16 tokens of a dimension.
// Probabilities never leave their lane; a query row stays in one lane (mod 16), so
// maxima and sums are the lane's own but for one exchange between lane groups where
// a reference changes, and one at the end.
//
// Codes become bf16 exactly, with their block's scale (a power of two): the
// keys' is folded into log2(e) * scale, the values' into the conversion.
//
// Two kernels (draft_plan says which, with both sides): split_kernel, whose waves
// have the same query rows, take different blocks straight from memory and join
// their sums at the end; and shared_kernel, whose waves have query rows of their own
// and share each block, converted once, in LDS.
//
// What bounds them (one MI355X):
//   64 requests x 32 heads (8 K/V) of 128, windows of 4096    97 us, 5.5 TB/s: HBM
//   one prompt chunk of 2048 tokens, the same heads and window  139 us, 990
//   TFLOP/s, 0.81 of a large bf16 product: by its counters the matrix units are
//   busy for 42 % of the cycles and vector instructions issue in 53 %; a matrix
//   instruction keeps the issue port for half of its time, so the two hardly
//   overlap
//   one request's token, window 1024   9 us: latency of 3 blocks a wave, which 8
//   compute units read
// (Tried for the prompt chunk: every wave on its own from memory 186 us, its
// loads a key apart; codes in LDS, converted by each wave, 146; with the
// exponentials beside the next block's products 154; 4 waves a workgroup 153.)
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

// The work of a workgroup: a share of the tokens for a tile of the query rows of
// an entry and head.  Workgroups are dealt to the 8 XCDs in turn: each XCD takes a
// run of neighbours, so that its L2 serves the tokens of one head to all of them.
struct Job {
    int i, kvh, tile, share;
    int64_t part;  // (entry, head, share)
};

__device__ __forceinline__ bool job_of(const AttendArgs &a, Job &j)
{
    const uint32_t job = (blockIdx.x & 7) * ((a.jobs + 7) / 8) + blockIdx.x / 8;
    if (job >= a.jobs)
        return false;
    j.share = (int)(job % (uint32_t)a.shares);
    const uint32_t rest = job / (uint32_t)a.shares;
    j.tile = (int)(rest % (uint32_t)a.tiles);
    const uint32_t unit = rest / (uint32_t)a.tiles;
    j.i = (int)(unit / (uint32_t)a.w.kv_heads);
    j.kvh = (int)(unit % (uint32_t)a.w.kv_heads);
    j.part = (int64_t)unit * a.shares + j.share;
    return true;
}

// Blocks of tokens that query rows [x0, x1) see, [b0, b1), and those that all of
// them see whole, [full0, full1).
struct Span {
    int b0, b1, full0, full1;
};

__device__ __forceinline__ Span span_of(const AttendArgs &a, const Entry &e, int x0, int x1)
{
    const int end0 = end_of(a.c.mask, e, x0 / a.group);
    const int end1 = end_of(a.c.mask, e, (x1 - 1) / a.group);
    const int lo0 = end0 > a.w.W ? end0 - a.w.W : 0, lo1 = end1 > a.w.W ? end1 - a.w.W : 0;
    return {lo0 / kBlock, (end1 + kBlock - 1) / kBlock, (lo1 + kBlock - 1) / kBlock,
            end0 / kBlock};
}

// A share of them.
__device__ __forceinline__ void cut(Span &s, int share, int shares)
{
    const int per = (s.b1 - s.b0 + shares - 1) / shares;
    s.b0 += share * per;
    s.b1 = s.b0 + per < s.b1 ? s.b0 + per : s.b1;
}

// A wave's query rows x0 .. x0 + 16 MB - 1 of an entry and head.
template <int D, int MB>
struct Rows {
    static constexpr int kSteps = D / 32;  // MFMA steps of a score
    static constexpr int kCols = D / 16;   // blocks of 16 value columns
    static constexpr int kKeys = D / 64;   // 16-byte pieces of a key in a lane
    typedef f32x4 Scores[4][MB];           // of a block's 4 tiles of 16 tokens
    frag q[MB][kSteps];
    int lo[MB], hi[MB];  // tokens that the lane's row of each block sees
    // m (0 before the first score), how far above it scores may be (-infinity
    // before the first), the lane's share of l
    float ref[MB], slack[MB], l[MB];
    f32x4 o[kCols][MB];
    u32x4 p[2][MB];  // probabilities: 8 tokens of each lane group in a frag

    // Rows past the last one are that row's, and not written.
    __device__ __forceinline__ void init(const AttendArgs &a, const Entry &e, int i, int kvh, int x0,
                                         int rows)
    {
        const int col = lane_id() & 15, grp = lane_id() >> 4;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int x = x0 + mb * 16 + col, xc = x < rows ? x : rows - 1;
            const int j = xc / a.group, h = kvh * a.group + xc % a.group;
            hi[mb] = end_of(a.c.mask, e, j);
            lo[mb] = hi[mb] > a.w.W ? hi[mb] - a.w.W : 0;
            const __bf16 *at = static_cast<const __bf16 *>(a.c.q) + i * a.c.q_stride_entry +
                               j * a.c.q_stride_query + h * a.c.q_stride_head;
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const __bf16 *from = at + st / 2 * 64 + grp * 16 + (st & 1) * 8;
                if (a.wide) {
                    q[mb][st] = *reinterpret_cast<const frag *>(from);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        q[mb][st][k] = from[k];
                }
                // a negative scale goes into the queries, so that the largest
                // product is the largest score
                if (a.c.scale < 0.f)
                    q[mb][st] = -q[mb][st];
            }
            ref[mb] = 0.f;
            slack[mb] = -__builtin_inff();
            l[mb] = 0.f;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                o[c][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }

    // Products with a block's keys: key(g) is the lane's operand of step g % kSteps of
    // tile g / kSteps.  Operands are asked for `AHEAD` steps early (fences keep it so).
    template <int AHEAD, typename K>
    __device__ __forceinline__ void scores(K key, Scores &s)
    {
        constexpr int N = 4 * kSteps;
        frag k[N];
#pragma unroll
        for (int g = 0; g < AHEAD; ++g)
            k[g] = key(g);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < N; ++g) {
            const int j = g / kSteps, st = g % kSteps;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                s[j][mb] = mfma(k[g], q[mb][st], st == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j][mb]);
            if (g + AHEAD < N)
                k[g + AHEAD] = key(g + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Leaves out the tokens of block b that a row does not see.
    __device__ __forceinline__ void mask(Scores &s, int b)
    {
        int first = b * kBlock + (lane_id() >> 4) * 16;
        asm("" : "+v"(first));  // (compared here, not ahead of the loop for each token)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t pos = (uint32_t)(first - lo[mb] + j * 4 + x);
                    if (pos >= (uint32_t)(hi[mb] - lo[mb]))
                        s[j][mb][x] = -__builtin_inff();
                }
    }

    // Scores relative to the reference, t - m, in place of the products (factor makes
    // t of one), and the lane's largest of each block of rows.
    __device__ __forceinline__ void relative(Scores &s, float factor, float (&top)[MB])
    {
#pragma unroll
        for (int e = 0; e < 8 * MB; ++e) {
            const int mb = e / 8, j = e / 2 % 4, x = e % 2 * 2;
            const float y0 = fmaf(s[j][mb][x], factor, -ref[mb]);
            const float y1 = fmaf(s[j][mb][x + 1], factor, -ref[mb]);
            s[j][mb][x] = y0;
            s[j][mb][x + 1] = y1;
            top[mb] = e % 8 == 0 ? fmaxf(y0, y1) : fmaxf(fmaxf(top[mb], y0), y1);
        }
    }

    // Where one is above the slack, the maximum becomes the reference.
    __device__ __forceinline__ void settle(Scores &s, const float (&top)[MB])
    {
        bool exceeds = false;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            exceeds |= top[mb] > slack[mb];
        if (!__any(exceeds))
            return;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            float by = fmaxf(top[mb], __shfl_xor(top[mb], 16));
            by = fmaxf(by, __shfl_xor(by, 32));
            if (slack[mb] == -__builtin_inff()) {  // none so far
                if (by == -__builtin_inff())
                    continue;
                slack[mb] = kSlack;
            } else {
                by = fmaxf(by, 0.f);
            }
            const float alpha = exp2_hw(-by);  // (finite sums of 0 stay 0 in the first case)
            ref[mb] += by;
            l[mb] = l[mb] == 0.f ? 0.f : l[mb] * alpha;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    o[c][mb][x] = o[c][mb][x] == 0.f ? 0.f : o[c][mb][x] * alpha;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j][mb] -= by;
        }
    }

    // Probabilities of a block, in pairs.
    __device__ __forceinline__ void probabilities(const Scores &s)
    {
#pragma unroll
        for (int e = 0; e < 8 * MB; ++e) {
            const int mb = e / 8, j = e / 2 % 4, x = e % 2 * 2;
            const float y0 = exp2_hw(s[j][mb][x]), y1 = exp2_hw(s[j][mb][x + 1]);
            l[mb] += y0;
            l[mb] += y1;
            // rounded to bf16 for the products (at most 2^-8 of it): the matrix
            // instruction takes 16 bits, and fp16, with three more, does not hold the
            // values times their block's scale; the sum and with it the lse take them
            // as they are.  Summed and rounded here, so that a pair takes one register
            // from now on
            uint32_t pair = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)y0, (__bf16)y1});
            asm volatile("" : "+v"(pair), "+v"(l[mb]));
            p[j / 2][mb][(j & 1) * 2 + x / 2] = pair;
        }
    }

    // Sums over a block's values: value(g) is the lane's operand of tokens 8 (g % 2) ..
    // of each 16, columns 16 (g / 2) ..; as in scores.
    template <int AHEAD, typename V>
    __device__ __forceinline__ void values(V value)
    {
        constexpr int N = 2 * kCols;
        frag v[N];
#pragma unroll
        for (int g = 0; g < AHEAD; ++g)
            v[g] = value(g);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < N; ++g) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                o[g / 2][mb] = mfma(v[g], __builtin_bit_cast(frag, p[g % 2][mb]), o[g / 2][mb]);
            if (g + AHEAD < N)
                v[g + AHEAD] = value(g + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // m of the sums.
    __device__ __forceinline__ float reference(int mb) const
    {
        return slack[mb] == -__builtin_inff() ? -__builtin_inff() : ref[mb];
    }

    // The lane groups' sums of probabilities.
    __device__ __forceinline__ void total()
    {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            l[mb] += __shfl_xor(l[mb], 16);
            l[mb] += __shfl_xor(l[mb], 32);
        }
    }
};

// What the products are multiplied by: log2(e) scale, and the keys' unit.  (At
// least a small normal: masked scores stay -infinity with a scale of 0.)
__device__ __forceinline__ float score_factor(float scale, uint32_t key_scale)
{
    return fmaxf(fabsf(scale) * 1.44269504088896340736f * scale_value(key_scale), 1e-37f);
}

// Row x of the head, columns d .. d + 3 of its unnormalised sums.
template <int D>
__device__ __forceinline__ void write_sums(const AttendArgs &a, const Job &job, int x, int d, float m,
                                           float l, f32x4 sums)
{
    if (a.shares > 1) {
        const int64_t at = job.part * (a.c.nq * a.group) + x;
        if (d == 0)
            *reinterpret_cast<float2 *>(a.stat + 2 * at) = make_float2(m, l);
        *reinterpret_cast<f32x4 *>(a.partial + at * D + d) = sums;
        return;
    }
    const int j = x / a.group, h = job.kvh * a.group + x % a.group;
    const int64_t at = ((int64_t)job.i * a.c.nq + j) * a.c.heads + h;
    const float inv = m == -__builtin_inff() && l == 0.f ? 0.f : 1.f / l;
    if (d == 0 && a.c.lse)
        a.c.lse[at] = 0.69314718055994530942f * (m + __log2f(l));
    bf16x4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        r[k] = (__bf16)(sums[k] * inv);
    *reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.c.out) + at * D + d) = r;
}

// Few query rows: the NW waves of a workgroup have the same ones and take every
// NW-th block of tokens, from memory into registers (the next keys once the scores
// are taken, the next values after the products); their sums are joined through LDS.
//
// A lane's pieces of a block's values, or of keys of 64, lie in whole lines that one
// load of the wave takes; those of longer keys would leave each line half read (some
// 20 bytes a cycle and compute unit), so keys of 128 and 256 are loaded in their order
// and change lanes through LDS: 8 K/V heads of 128 of one request, window 1024, 8.9
// us (10.6 without), 1024 tokens 94 (102), but 16 requests of 16 queries x 4 heads 25
// (24); values as well 9.2, keys of 64 as well 10.0 (9.6: 32 requests of 4 queries).
template <int D, int MB, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
void split_kernel(AttendArgs a)
{
    typedef Rows<D, MB> R;
    constexpr int kRows = 16 * MB, kStride = D + 4;
    constexpr int kPieces = D / 16;  // of a key, and of a lane in a block's keys or values
    constexpr bool kTurn = D >= 128;
    // 16-byte pieces of a key lie at piece ^ this, so that the 8 keys which a lane
    // group reads at once (key_at + 4 j, below) are in different banks
    auto key_swizzle = [](int t) { return (t & 3) | (t >> 2 & 4); };
    // a wave's keys; at the end the waves' sums
    __shared__ __attribute__((aligned(128))) float sO[NW * kRows * kStride];
    static_assert(!kTurn || sizeof(sO) >= NW * kBlock * D, "a block for each wave");
    __shared__ float sStat[NW * kRows * 2];
    const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    Job job;
    if (!job_of(a, job))
        return;
    const Entry e = attend_entry(a, job.i);
    if (a.c.status && job.kvh == 0 && job.tile == 0 && job.share == 0 && threadIdx.x == 0)
        a.c.status[job.i] = e.status;
    const int x0 = job.tile * kRows, rows = e.count * a.group;
    if (e.status != KVR_OK || x0 >= rows)
        return;
    Span span = span_of(a, e, x0, x0 + kRows < rows ? x0 + kRows : rows);
    cut(span, job.share, a.shares);
    R r;
    r.init(a, e, job.i, job.kvh, x0, rows);

    u32x4 k[kPieces], v[kPieces];
    uint32_t k_scale = 0, v_scale = 0;
    const int64_t head_bytes = 2 * kBlock * D;
    const int64_t first = (int64_t)e.r * a.w.blocks * a.w.kv_heads + job.kvh;
    // the lane's operands are pieces n of keys key_at + 4 j, and of values 16 c + col
    const int key_at = (col >> 2) * 16 + (col & 3);
    uint8_t *tile = reinterpret_cast<uint8_t *>(sO) + wave * (kBlock * D);
    auto at_block = [&](int b) { return first + (int64_t)(b % a.w.blocks) * a.w.kv_heads; };
    auto load_keys = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t *from = a.w.codes + at * head_bytes;
#pragma unroll
        for (int n = 0; n < kPieces; ++n)
            k[n] = *reinterpret_cast<const u32x4 *>(
                from + (kTurn ? n * 1024 + lane * 16
                              : (key_at + n / R::kKeys * 4) * D + (n % R::kKeys * 4 + grp) * 16));
        k_scale = a.w.scales[at * 2];
    };
    auto load_values = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t *from = a.w.codes + at * head_bytes + kBlock * D + col * kBlock + grp * 16;
#pragma unroll
        for (int c = 0; c < R::kCols; ++c)
            v[c] = *reinterpret_cast<const u32x4 *>(from + c * 16 * kBlock);
        v_scale = a.w.scales[at * 2 + 1];
    };
    int b = span.b0 + wave;
    if (b < span.b1) {
        load_keys(at_block(b));
        load_values(at_block(b));
    }
    for (; b < span.b1; b += NW) {
        typename R::Scores s;
        float top[MB];
        u32x4 turned[kTurn ? kPieces : 1];
        if constexpr (kTurn) {
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                const int t = (n * 64 + lane) / kPieces, piece = lane % kPieces;
                *reinterpret_cast<u32x4 *>(tile + t * D + (piece ^ key_swizzle(t)) * 16) = k[n];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                const int t = key_at + n / R::kKeys * 4, piece = n % R::kKeys * 4 + grp;
                turned[n] =
                    *reinterpret_cast<const u32x4 *>(tile + t * D + (piece ^ key_swizzle(t)) * 16);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        r.template scores<1>(
            [&](int g) __attribute__((always_inline)) {
                const int n = g / 2, half = g % 2 * 2;
                const u32x4 w = kTurn ? turned[kTurn ? n : 0] : k[n];
                return widen(w[half], w[half + 1], 1.f);
            },
            s);
        const float factor = score_factor(a.c.scale, k_scale);
        const bool more = b + NW < span.b1;
        const int64_t at_next = at_block(b + NW);
        if (more)
            load_keys(at_next);
        if (b < span.full0 || b >= span.full1)
            r.mask(s, b);
        r.relative(s, factor, top);
        r.settle(s, top);
        r.probabilities(s);
        const float unit = scale_value(v_scale);
        r.template values<1>(
            [&](int g) __attribute__((always_inline)) {
                return widen(v[g / 2][g % 2 * 2], v[g / 2][g % 2 * 2 + 1], unit);
            });
        if (more)
            load_values(at_next);
    }

    if constexpr (kTurn)
        __syncthreads();  // (the sums take the tiles' place)
    r.total();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int at = wave * kRows + mb * 16 + col;
        if (grp == 0) {
            sStat[at * 2] = r.reference(mb);
            sStat[at * 2 + 1] = r.l[mb];
        }
#pragma unroll
        for (int c = 0; c < R::kCols; ++c)
            *reinterpret_cast<f32x4 *>(&sO[at * kStride + c * 16 + grp * 4]) = r.o[c][mb];
    }
    __syncthreads();
    // the waves' sums, joined in wave order
    for (int q = threadIdx.x; q < kRows * D / 4; q += NW * 64) {
        const int row = q / (D / 4), d = q % (D / 4) * 4;
        if (x0 + row >= rows)
            break;
        float m = -__builtin_inff(), l = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            m = fmaxf(m, sStat[(w * kRows + row) * 2]);
        f32x4 sums = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int at = w * kRows + row;
            const float mw = sStat[at * 2], lw = sStat[at * 2 + 1];
            // (a wave without a score above -infinity has sums of 0 or NaN)
            const float weight = mw == -__builtin_inff() ? 1.f : exp2_hw(mw - m);
            l += weight * lw;
            sums += weight * *reinterpret_cast<const f32x4 *>(&sO[at * kStride + d]);
        }
        write_sums<D>(a, job, x0 + row, d, m, l, sums);
    }
}

// A workgroup barrier for LDS: loads from memory stay in flight.
__device__ __forceinline__ void barrier_lds()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Many query rows: the NW waves of a workgroup have some each and share the blocks
// of tokens, of which each converts its part to bf16 (the values with their
// scale), once for all, into LDS.
//
// While one block is worked on, the next is converted into the other half of LDS,
// and the codes of the one after it are on their way.
//
// 16-byte pieces lie at piece ^ swizzle of their row: keys in rows 16 a + 4 j + b (a,
// b = 0 .. 3) of 2 D bytes, values in 16 consecutive rows of 128.  The keys are read
// without bank conflicts.  Reads of the values take twice their time, 4 cycles more
// each, and the stores of both 8 more (each pattern counted alone): with heads of 128 96
// of the 256 LDS cycles of a wave and block.
template <int D, int MB, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(NW / 4)))
void shared_kernel(AttendArgs a)
{
    typedef Rows<D, MB> R;
    constexpr int kPart = kBlock * D / NW / 16;       // 16-code pieces of a wave, keys or values
    constexpr int kLoads = kPart / 64;
    static_assert(D >= 128 && kPart % 64 == 0, "every lane has pieces, keys take 4 steps or more");
    constexpr int kHalf = 2 * kBlock * D;             // bytes of a block's keys or values
    __shared__ __attribute__((aligned(1024))) uint8_t sTile[2][2 * kHalf];  // keys, values
    const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    Job job;
    if (!job_of(a, job))
        return;
    const Entry e = attend_entry(a, job.i);
    if (a.c.status && job.kvh == 0 && job.tile == 0 && job.share == 0 && threadIdx.x == 0)
        a.c.status[job.i] = e.status;
    const int rows = e.count * a.group;
    const int first_row = job.tile * NW * 16 * MB;  // of the workgroup, and of the wave
    if (e.status != KVR_OK || first_row >= rows)
        return;
    const int x0 = first_row + wave * 16 * MB;
    auto below = [&](int x) { return x < rows ? x : rows; };
    Span all = span_of(a, e, first_row, below(first_row + NW * 16 * MB));
    cut(all, job.share, a.shares);
    const bool idle = x0 >= rows;
    const Span own = span_of(a, e, idle ? rows - 1 : x0, below(x0 + 16 * MB));
    R r;
    r.init(a, e, job.i, job.kvh, idle ? rows - 1 : x0, rows);

    auto key_swizzle = [](int row) { return (row >> 4 & 3) * 4 + (row & 3); };
    auto value_swizzle = [](int row) { return row >> 1 & 7; };
    const int64_t first = (int64_t)e.r * a.w.blocks * a.w.kv_heads + job.kvh;
    // (past the last block: that one's again, not used)
    auto at_block = [&](int b) {
        return first + (int64_t)((b < all.b1 ? b : all.b1 - 1) % a.w.blocks) * a.w.kv_heads;
    };
    // The lane's pieces of a block: codes from `from`, bf16 values to the two `to`.
    u32x4 k_raw[kLoads], v_raw[kLoads];
    uint32_t k_scale = 0, v_scale = 0;
    int from[kLoads], k_to[kLoads][2], v_to[kLoads][2];
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
        const int piece = wave * kPart + n * 64 + lane;
        const int key = piece / (D / 16), value = piece / 4;
        from[n] = piece * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            k_to[n][h] = key * 2 * D + ((piece % (D / 16) * 2 + h) ^ key_swizzle(key)) * 16;
            v_to[n][h] = kHalf + value * 128 + ((piece % 4 * 2 + h) ^ value_swizzle(value)) * 16;
        }
    }
    auto load = [&](int b) __attribute__((always_inline)) {
        const int64_t at = at_block(b);
        const uint8_t *codes = a.w.codes + at * (2 * kBlock * D);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            k_raw[n] = *reinterpret_cast<const u32x4 *>(codes + from[n]);
            v_raw[n] = *reinterpret_cast<const u32x4 *>(codes + kBlock * D + from[n]);
        }
        k_scale = a.w.scales[at * 2];
        v_scale = a.w.scales[at * 2 + 1];
    };
    uint32_t next_scale = 0;  // of the keys of the block stored last
    auto store = [&](uint8_t *to) __attribute__((always_inline)) {
        const float unit = scale_value(v_scale);
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                *reinterpret_cast<frag *>(to + k_to[n][h]) =
                    widen(k_raw[n][h * 2], k_raw[n][h * 2 + 1], 1.f);
                *reinterpret_cast<frag *>(to + v_to[n][h]) =
                    widen(v_raw[n][h * 2], v_raw[n][h * 2 + 1], unit);
            }
        next_scale = k_scale;
    };
    int k_at[4], v_at[2];
#pragma unroll
    for (int st = 0; st < 4; ++st) {
        const int row = (col >> 2) * 16 + (col & 3);
        k_at[st] = row * 2 * D + ((st / 2 * 8 + grp * 2 + st % 2) ^ key_swizzle(row)) * 16;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        v_at[h] = kHalf + col * 128 + ((grp * 2 + h) ^ value_swizzle(col)) * 16;

    int t = all.b0;  // the block that is worked on next
    if (t < all.b1) {
        load(t);
        store(sTile[t & 1]);
        load(t + 1);
    }
    float factor = 0.f;
    auto next = [&]() __attribute__((always_inline)) {
        barrier_lds();
        factor = score_factor(a.c.scale, next_scale);
        ++t;
        store(sTile[t & 1]);
        load(t + 1);
    };
    // (blocks that this wave's rows do not see come before and after those that
    // they do)
    const int b0 = idle || own.b0 > all.b1 ? all.b1 : own.b0;
    const int b1 = own.b1 < all.b1 ? own.b1 : all.b1;
    while (t < b0)
        next();
    for (int b = t; b < b1; ++b) {
        next();
        typename R::Scores s;
        float top[MB];
        const uint8_t *tile = sTile[b & 1];
        r.template scores<4>(
            [&](int g) __attribute__((always_inline)) {
                const int j = g / R::kSteps, st = g % R::kSteps;
                return *reinterpret_cast<const frag *>(tile + k_at[st % 4] + st / 4 * 256 +
                                                       j * 8 * D);
            },
            s);
        if (b < own.full0 || b >= own.full1)
            r.mask(s, b);
        r.relative(s, factor, top);
        r.settle(s, top);
        r.probabilities(s);
        r.template values<4>(
            [&](int g) __attribute__((always_inline)) {
                return *reinterpret_cast<const frag *>(tile + v_at[g % 2] + g / 2 * 16 * 128);
            });
    }
    while (t < all.b1)
        next();
    r.total();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int x = x0 + mb * 16 + col;
        if (x >= rows)
            continue;
#pragma unroll
        for (int c = 0; c < R::kCols; ++c)
            write_sums<D>(a, job, x, c * 16 + grp * 4, r.reference(mb), r.l[mb], r.o[c][mb]);
    }
}

// Joins the shares of each query row: a workgroup per row, its waves taking
// every fourth share, their sums added in wave order; or, of the thousands of rows
// that shared_kernel leaves, a wave per row.  Bound by launch and latency (32 rows of
// 128 in 8 shares 4.2 us), or by reading the shares (16384 rows of 256 in two 10.5
// us, with a workgroup per row 23.5; of few rows a wave per row is slower, 4 requests
// of 32 heads in 8 shares 15.5 us in all against 14.3).
constexpr int kJoinWaves = 4;
template <int D, int PER>  // waves of a row
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(AttendArgs a)
{
    constexpr int N = D / 64;   // columns of a lane
    constexpr int kFlight = 4;  // shares in flight
    typedef float vec __attribute__((ext_vector_type(N)));
    __shared__ float sL[kJoinWaves];
    __shared__ vec sO[kJoinWaves][64];
    const int lane = lane_id(), wave = wave_id() % PER;
    const int unit_rows = a.c.nq * a.group;
    const uint32_t at_row = blockIdx.x * (kJoinWaves / PER) + wave_id() / PER;
    const uint32_t unit = at_row / (uint32_t)unit_rows;
    const int x = (int)(at_row % (uint32_t)unit_rows);
    const int i = (int)(unit / (uint32_t)a.w.kv_heads), kvh = (int)(unit % (uint32_t)a.w.kv_heads);
    if (i >= a.c.n)
        return;
    const Entry e = attend_entry(a, i);
    const int j = x / a.group, h = kvh * a.group + x % a.group;
    if (e.status != KVR_OK || j >= e.count)
        return;
    const int64_t first = (int64_t)unit * a.shares * unit_rows + x;
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
    for (int s0 = wave; s0 < a.shares; s0 += PER * kFlight) {
        vec part[kFlight];
        float w[kFlight], ls[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int s = s0 + f * PER;
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
    if constexpr (PER > 1) {
        sO[wave][lane] = o;
        if (lane == 0)
            sL[wave] = l;
        __syncthreads();
        if (wave != 0)
            return;
#pragma unroll
        for (int k = 1; k < PER; ++k) {
            l += sL[k];
            o += sO[k][lane];
        }
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

// A wave's blocks of 16 query rows where there are many: as many as two waves a SIMD
// have registers for.
constexpr int split_rows(int d) { return d == 256 ? 1 : 2; }

// Waves that share a block in LDS, each with 32 query rows (with heads of 256 they
// need more than half of a SIMD's registers).
constexpr int shared_waves(int d) { return d == 256 ? 4 : 8; }

int64_t partial_bytes(int64_t rows, int32_t d) { return rows * (d + 2) * (int64_t)sizeof(float); }

template <int D>
hipError_t launch_dim(const AttendArgs &a, const DraftPlan &p, dim3 grid, hipStream_t s)
{
    auto run = [&](void (*kernel)(AttendArgs), int waves) {
        return launch(nullptr, 0, kernel, grid, dim3(waves * 64), 0, s, a);
    };
    hipError_t e;
    if constexpr (D == 64)
        e = p.blocks_of_16 == 2 ? run(split_kernel<D, 2, 4>, 4)
            : p.waves == 4      ? run(split_kernel<D, 1, 4>, 4)
                                : run(split_kernel<D, 1, 8>, 8);
    else if constexpr (D == 128)
        e = !p.split              ? run(shared_kernel<D, 2, 8>, 8)
            : p.blocks_of_16 == 2 ? run(split_kernel<D, 2, 4>, 4)
            : p.waves == 4        ? run(split_kernel<D, 1, 4>, 4)
                                  : run(split_kernel<D, 1, 8>, 8);
    else
        e = !p.split ? run(shared_kernel<D, 2, 4>, 4) : run(split_kernel<D, 1, 4>, 4);
    if (e != hipSuccess || a.shares == 1)
        return e;
    const int64_t rows = (int64_t)a.c.n * a.c.nq * a.c.heads;
    // (heads of 256 are the only ones whose shared_kernel makes shares; of 128, windows of
    // 4096, in two: 512 tokens 99 us, split 50; 1024 121, 92; 2400 317, 210)
    if constexpr (D == 256)
        if (!p.split)
            return launch(nullptr, 0, join_kernel<D, 1>,
                          dim3((unsigned)((rows + kJoinWaves - 1) / kJoinWaves)),
                          dim3(kJoinWaves * 64), 0, s, a);
    return launch(nullptr, 0, join_kernel<D, kJoinWaves>, dim3((unsigned)rows),
                  dim3(kJoinWaves * 64), 0, s, a);
}

}  // namespace

DraftPlan draft_plan(int32_t n, int32_t nq, int32_t heads, int32_t kv_heads, int32_t d_head,
                     int32_t tokens)
{
    DraftPlan p{};
    const int64_t rows = (int64_t)nq * (heads / kv_heads);  // of an entry and head
    const int64_t units = (int64_t)n * kv_heads;
    const int64_t blocks = ((int64_t)tokens + kBlock - 1) / kBlock + 1;
    // shared_kernel takes whole rounds of the compute units (256 query rows a
    // workgroup, with heads of 256 128).  Heads of 128, windows of 4096: a chunk of 1024
    // tokens (128 workgroups) 134 us against 92 split, 1500 (188) 135, 134, 1700 (213)
    // 136, 155, 2048 (256) 139, 177, 2400 (300) 262, 210, 3000 (375) 263, 259: so with
    // 0.75 of its rounds full.  Heads of 256, whose shares fill a part of one round: 256
    // tokens (32 workgroups, one round of the other kernel) 53, 46, 300 (40) 58, 85, 512
    // (64) 78, 89, with windows of 1024 41, 37, 1024 (128) 128, 172; 2400 (300) 415, 414,
    // 2700 (340) 415, 457: so past an eighth, and past one round with 0.6.  Heads of 64,
    // for which it is not built, lose by it with long windows (64 heads, windows of
    // 4096: 512 tokens 99, split 53; 1024, a full round, 101, 98; 2048 198, 185; 4096 390,
    // 360; 1000 of 56 heads, windows of 2000, 57, 51) and would gain by full rounds
    // and short ones (windows of 1024: 1024 tokens 36, 39, 2048 68, 70; of 256: 34, 43).
    const int64_t shared = 16 * 2 * shared_waves(d_head);
    const int64_t full = units * ((rows + shared - 1) / shared);
    const int64_t room = (full + kUnits - 1) / kUnits * kUnits;
    p.split = d_head == 64 || rows < shared ||
              (d_head == 128    ? 4 * full < 3 * room
               : full <= kUnits ? 8 * full <= kUnits
                                : 5 * full < 3 * room);
    // (blocks of 16 while that leaves no workgroup waiting: 8 requests of 8 queries
    // x 4 heads, windows of 1024, 11 us, in blocks of 32 17; 64 requests of 5 38, 34)
    p.blocks_of_16 = !p.split ? 2
                     : rows <= 16 || units * ((rows + 15) / 16) <= kUnits ? 1
                                                                          : split_rows(d_head);
    const int64_t tile = p.split ? 16 * p.blocks_of_16 : shared;
    p.tiles = (int32_t)((rows + tile - 1) / tile);
    const int64_t groups = units * p.tiles;
    p.waves = !p.split ? shared_waves(d_head) : d_head == 256 || groups > kUnits ? 4 : 8;
    if (p.split && p.blocks_of_16 == 2)
        p.waves = 4;
    // (8 waves where there are few workgroups: 32 requests of 4 queries x 7 heads of 64
    // 10 us, with 4 waves 12; 512 workgroups, window 256: 15, 12)
    // Shares where there are three or more and they take 24 blocks of 16 KB off a
    // workgroup, which pays for the join (8 K/V heads, windows of 4096): one request 18
    // us in one share, 11 in 8; 8 requests 20, 19 in 4; 16 requests 31, 34 in 2; windows
    // of 2048: one 11.8, 10.5 in 4; of 1024: 8.8, 9.8 in 4.
    int64_t shares = kUnits / groups;
    shares = shares < blocks / p.waves ? shares : blocks / p.waves;
    if (shares < (p.split ? 3 : 2) || (blocks - blocks / shares) * d_head < 24 * 128)
        shares = 1;
    p.shares = (int32_t)shares;
    p.workspace = p.shares > 1 ? partial_bytes(units * p.shares * rows, d_head) : 0;
    return p;
}

// Over all smaller calls: their query rows times shares are at most the query
// rows times the most shares, and at most the rows of 256 workgroups.
int64_t draft_workspace_bound(int32_t n, int32_t nq, int32_t heads, int32_t kv_heads,
                              int32_t d_head, int32_t window)
{
    const int64_t blocks = ((int64_t)window + nq - 1 + kBlock - 1) / kBlock + 1;
    const int64_t most = blocks / 4, all = (int64_t)n * nq * heads;
    const int64_t tile = 16 * 2 * shared_waves(d_head);
    (void)kv_heads;
    if (most < 2)
        return 0;
    return partial_bytes(all * most < kUnits * tile ? all * most : kUnits * tile, d_head);
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
