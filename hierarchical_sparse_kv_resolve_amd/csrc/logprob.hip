// Log probabilities of given tokens, entropy and the most likely alternatives
// of rows of logits ("Adaptive DHiSparse: Speculative Decoding over a
// Load-Adaptive KV Hierarchy", section "How it works", paragraph "Speculative
// state": verification scores the drafted tokens).
//
// With m the row's largest logit, f = log2(e) * scale and d_j = f (x_j - m) <= 0
// (the difference first, so that logits of the type's lowest value do not
// overflow):
//   l = sum 2^d_j,  u = -sum 2^d_j d_j   (terms >= 0: nothing cancels)
//   lse = scale m + ln l,  entropy = ln l + ln 2 u / l
//   logprob = scale (x - m) - ln l
//
// part_kernel reads the logits once: a row is cut into shares of a workgroup
// each, whose threads keep m, l, u and their largest logit.
// row_kernel, a workgroup per row, joins the shares.  For the alternatives it
// takes the threads' largest logits in 128 groups (every 128th piece): the top-th
// largest of the groups' maxima is a value that at least `top` logits reach,
// so only the runs of threads whose maximum reaches it are read again, and of
// those logits the few that reach it are ranked by counting, (value, lower token
// first), which needs no order of arrival.  Rows with so many that the list
// overflows (equal logits, or large ones that all fell to one group) are
// searched once for each alternative instead.
//
// What they take (one MI355X, 131072 bf16 logits, 20 alternatives): 128 rows 11 us, by
// its counters bound by the issue of vector instructions (14 a logit, in three quarters
// of its cycles; reading 34 MB alone would take 7; the entropy's part is paid without
// one as well), and 7 to 8; one row 3.5 and 6.9, the latency of reading the maxima, of
// three barriers and of reading the runs that reach the bound.  64 alternatives of
// 64 rows take 8.1 and 10.5 (with 64 groups, of whose maxima the 64th bounds next to
// nothing, the list overflowed: 190 in all).  128 rows with 8 pieces of a thread in
// flight 20.1 in all, with 4 18.7.
#include "block.h"
#include "kvr_internal.h"
#include "values.h"

namespace kvr {
namespace {

constexpr int NT = 256;
constexpr int kRun = 8;        // consecutive logits of a thread: one piece
constexpr int kBatch = 4;      // pieces of a thread in flight
constexpr int kList = 1024;    // logits that are ranked, and runs that are read for them
constexpr float kInf = __builtin_inff();

struct LogprobArgs {
    kvr_logprob_call c;
    int32_t shares, pieces;  // of a row
    int32_t per;             // pieces of a share (a multiple of NT, but for the last)
    bool wide;
    float *parts;            // [n][shares][4]: m, l, u
    float *tops;             // [n][shares][NT]: the threads' largest logits
};

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Logits [8 piece, 8 piece + 8) of a row, -infinity past its end.
template <typename T>
__device__ __forceinline__ void load_piece(const LogprobArgs &a, const T *row, int piece,
                                           float (&x)[kRun])
{
    const int at = piece * kRun;
    if (at + kRun <= a.c.vocab) {
        load_run<kRun>(row + at, a.wide, x);
    } else {
#pragma unroll
        for (int k = 0; k < kRun; ++k)
            x[k] = at + k < a.c.vocab ? (float)row[at + k] : -kInf;
    }
}

// Moves l and u to the reference `to` >= m: what m rises by is added to u for
// each probability.  m may be -infinity (l is 0 then, or NaN).
__device__ __forceinline__ void raise(float factor, float m, float &l, float &u, float to)
{
    const float d = (m - to) * factor;  // NaN for two infinities of one sign
    const float w = exp2_hw(m == -kInf ? -kInf : d);
    u = w > 0.f ? w * (u - d * l) : 0.f;
    l *= w;
}

// Joins (m, l, u) of another part.
__device__ __forceinline__ void join(float factor, float &m, float &l, float &u, float m2, float l2,
                                     float u2)
{
    const float to = fmaxf(m, m2);
    raise(factor, m, l, u, to);
    raise(factor, m2, l2, u2, to);
    m = to;
    l += l2;
    u += u2;
}

template <typename T>
__global__ __launch_bounds__(NT) void part_kernel(LogprobArgs a)
{
    __shared__ float sM[NT / 64], sL[NT / 64], sU[NT / 64];
    const int64_t row_at = blockIdx.x / a.shares;
    const int share = blockIdx.x % a.shares;
    const T *row = static_cast<const T *>(a.c.logits) + row_at * a.c.logits_stride;
    const int p0 = share * a.per;
    const int p1 = p0 + a.per < a.pieces ? p0 + a.per : a.pieces;
    const float factor = a.c.scale * 1.44269504088896340736f;
    float m = -kInf, l = 0.f, u = 0.f;
    auto add = [&](auto &x) __attribute__((always_inline)) {  // [pieces][kRun]
        float to = m;
#pragma unroll
        for (auto &piece : x)
#pragma unroll
            for (float y : piece)
                to = fmaxf(to, y);
        raise(factor, m, l, u, to);
        m = to;
        const float ref = to == -kInf ? 0.f : to;
#pragma unroll
        for (auto &piece : x)
#pragma unroll
            for (float y : piece) {
                const float d = (y - ref) * factor;
                const float e = exp2_hw(d);
                l += e;
                u -= e > 0.f ? e * d : 0.f;
            }
    };
    int p = p0 + threadIdx.x;
    for (; p + (kBatch - 1) * NT < p1; p += kBatch * NT) {
        float x[kBatch][kRun];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            load_piece(a, row, p + k * NT, x[k]);
        add(x);
    }
    for (; p < p1; p += NT) {
        float x[1][kRun];
        load_piece(a, row, p, x[0]);
        add(x);
    }
    if (a.c.top > 0)
        a.tops[(int64_t)blockIdx.x * NT + threadIdx.x] = m;
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1)
        join(factor, m, l, u, __shfl_xor(m, k), __shfl_xor(l, k), __shfl_xor(u, k));
    if (lane_id() == 0) {
        sM[wave_id()] = m;
        sL[wave_id()] = l;
        sU[wave_id()] = u;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int k = 1; k < NT / 64; ++k)
            join(factor, m, l, u, sM[k], sL[k], sU[k]);
        float *out = a.parts + (int64_t)blockIdx.x * 4;
        out[0] = m;
        out[1] = l;
        out[2] = u;
    }
}

// (x, i) before (y, j): larger, or equal and lower.
__device__ __forceinline__ bool before(float x, int i, float y, int j)
{
    return x > y || (x == y && i < j);
}

// Floats as integers of the same order.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// The n-th largest of the 64 lanes' two values, bit by bit from the top.
__device__ __forceinline__ float nth_largest(float x, float y, int n)
{
    const uint32_t kx = key_of(x), ky = key_of(y);
    uint32_t found = 0;
#pragma unroll
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t trial = found | 1u << bit;
        if (__popcll(__ballot(kx >= trial)) + __popcll(__ballot(ky >= trial)) >= n)
            found = trial;
    }
    return __uint_as_float(found ^ (found >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// NR threads a row, TOPS maxima of the threads before in each at once.
template <typename T, int NR, int TOPS>
__global__ __launch_bounds__(NR) void row_kernel(LogprobArgs a)
{
    constexpr int kWaves = NR / 64;
    __shared__ float sMost[kWaves][64];
    __shared__ float sValue[kList];
    __shared__ int sToken[kList];
    __shared__ int sRun[kList];
    __shared__ int sRuns, sCount;
    __shared__ float sSum[2];  // m and ln l (NaN where anything is)
    __shared__ float sM[kWaves];
    __shared__ int sI[kWaves];
    const int64_t r = blockIdx.x;
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const T *row = static_cast<const T *>(a.c.logits) + r * a.c.logits_stride;
    const float factor = a.c.scale * 1.44269504088896340736f;
    if (tid == 0)
        sRuns = sCount = 0;

    const int top = a.c.top;
    const int runs = top > 0 ? a.shares * NT : 0;
    const float *tops = a.tops + r * a.shares * NT;
    float t[TOPS];
#pragma unroll
    for (int k = 0; k < TOPS; ++k)
        t[k] = tid + k * NR < runs ? tops[tid + k * NR] : -kInf;

    // The last wave joins the row's sums, in a fixed order, and writes what needs no
    // more than them: beside the other waves' reads, below.
    constexpr float kLn2 = 0.69314718055994530942f;
    auto logprob = [&](float x, float m, float log_l) {
        return log_l != log_l ? log_l : x == -kInf ? -kInf : (x - m) * a.c.scale - log_l;
    };
    auto logit = [&](int k) {
        const int token = a.c.tokens[r * a.c.m + k];
        return token >= 0 && token < a.c.vocab ? (float)row[token] : -kInf;
    };
    auto sums = [&]() {
        if (wave != kWaves - 1)
            return;
        const float given = lane < a.c.m ? logit(lane) : 0.f;
        float m = -kInf, l = 0.f, u = 0.f;
        const float *parts = a.parts + r * a.shares * 4;
        for (int s = lane; s < a.shares; s += 64)
            join(factor, m, l, u, parts[4 * s], parts[4 * s + 1], parts[4 * s + 2]);
#pragma unroll
        for (int k = 32; k >= 1; k >>= 1)
            join(factor, m, l, u, __shfl_xor(m, k), __shfl_xor(l, k), __shfl_xor(u, k));
        // the first lane's, for all: the lanes' sums differ in their last bits (their
        // products are not fused alike)
        auto first = [](float x) {
            return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
        };
        m = first(m), l = first(l), u = first(u);
        const bool bad = l != l;  // a NaN, or an infinity
        const float log_l = bad ? __builtin_nanf("") : kLn2 * __log2f(l);
        if (lane == 0) {
            sSum[0] = m;
            sSum[1] = log_l;
            if (a.c.lse)
                a.c.lse[r] = bad ? log_l : m == -kInf ? -kInf : m * a.c.scale + log_l;
            if (a.c.entropy)
                a.c.entropy[r] = bad ? log_l : m == -kInf ? 0.f : log_l + kLn2 * (u / l);
        }
        if (lane < a.c.m)
            a.c.logprob[r * a.c.m + lane] = logprob(given, m, log_l);
    };
    // Given tokens past the 64th, once the sums are there.
    auto others = [&]() {
        for (int k = 64 + tid; k < a.c.m; k += NR)
            a.c.logprob[r * a.c.m + k] = logprob(logit(k), sSum[0], sSum[1]);
    };
    if (top == 0) {
        sums();
        __syncthreads();
        others();
        return;
    }
    int32_t *ids = a.c.top_ids + r * top;
    float *probs = a.c.top_logprob + r * top;

    // the maxima of 128 groups (a lane of the even or the odd waves)
    float most = -kInf;
#pragma unroll
    for (int k = 0; k < TOPS; ++k)
        most = fmaxf(most, t[k]);
    for (int q = tid + TOPS * NR; q < runs; q += NR)
        most = fmaxf(most, tops[q]);
    sMost[wave][lane] = most;
    __syncthreads();
    float even = -kInf, odd = -kInf;
#pragma unroll
    for (int k = 0; k < kWaves; k += 2) {
        even = fmaxf(even, sMost[k][lane]);
        odd = fmaxf(odd, sMost[k + 1][lane]);
    }
    const float bound = nth_largest(even, odd, top);  // (uniform: the same in every wave)
    auto keep = [&](int q, float x) __attribute__((always_inline)) {
        if (x >= bound && x > -kInf) {
            const int n = atomicAdd(&sRuns, 1);
            if (n < kList)
                sRun[n] = q;
        }
    };
#pragma unroll
    for (int k = 0; k < TOPS; ++k)
        keep(tid + k * NR, t[k]);
    for (int q = tid + TOPS * NR; q < runs; q += NR)
        keep(q, tops[q]);
    __syncthreads();
    const int found = sRuns;
    const int each = a.per / NT;  // pieces of a run
    if (found <= kList)
        for (int q = tid; q < found * each; q += NR) {
            const int run = sRun[q / each], s = run / NT;
            const int p = s * a.per + q % each * NT + run % NT;
            const int p1 = (s + 1) * a.per < a.pieces ? (s + 1) * a.per : a.pieces;
            if (p >= p1)
                continue;
            float x[kRun];
            load_piece(a, row, p, x);
#pragma unroll
            for (int k = 0; k < kRun; ++k)
                if (x[k] >= bound && x[k] > -kInf) {
                    const int n = atomicAdd(&sCount, 1);
                    if (n < kList) {
                        sValue[n] = x[k];
                        sToken[n] = p * kRun + k;
                    }
                }
        }
    sums();
    __syncthreads();
    others();
    const float m = sSum[0], log_l = sSum[1];
    if (log_l != log_l || m == -kInf) {
        if (tid < top) {
            ids[tid] = -1;
            probs[tid] = log_l != log_l ? log_l : -kInf;
        }
        return;
    }
    const int count = sCount;
    if (found <= kList && count <= kList) {
        // a wave ranks a logit at a time, its lanes holding the others
        for (int n = wave; n < count; n += kWaves) {
            const float x = sValue[n];
            const int token = sToken[n];
            int rank = 0;
            for (int k = lane; k < count + 63 - (count + 63) % 64; k += 64)
                rank += __popcll(__ballot(k < count && before(sValue[k], sToken[k], x, token)));
            if (rank < top && lane == 0) {
                ids[rank] = token;
                probs[rank] = logprob(x, m, log_l);
            }
        }
        for (int k = count + tid; k < top; k += NR) {  // fewer than asked for
            ids[k] = -1;
            probs[k] = -kInf;
        }
        return;
    }
    // too many reach the bound: one search of the row for each alternative
    float last = kInf;
    int last_token = -1;
    for (int k = 0; k < top; ++k) {
        float x = -kInf;
        int token = a.c.vocab;
        for (int p = tid; p < a.pieces; p += NR) {
            float y[kRun];
            load_piece(a, row, p, y);
#pragma unroll
            for (int q = 0; q < kRun; ++q)
                if (before(last, last_token, y[q], p * kRun + q) &&
                    before(y[q], p * kRun + q, x, token)) {
                    x = y[q];
                    token = p * kRun + q;
                }
        }
#pragma unroll
        for (int q = 32; q >= 1; q >>= 1) {
            const float y = __shfl_xor(x, q);
            const int other = __shfl_xor(token, q);
            if (before(y, other, x, token)) {
                x = y;
                token = other;
            }
        }
        if (lane == 0) {
            sM[wave] = x;
            sI[wave] = token;
        }
        __syncthreads();
        x = sM[0];
        token = sI[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            if (before(sM[w], sI[w], x, token)) {
                x = sM[w];
                token = sI[w];
            }
        __syncthreads();
        if (tid == 0) {
            ids[k] = x == -kInf ? -1 : token;
            probs[k] = logprob(x, m, log_l);
        }
        last = x;
        last_token = token;
    }
}

// Shares of a row in which a thread has `pieces` pieces.
int64_t shares_with(int32_t vocab, int pieces)
{
    return ((int64_t)vocab + kRun * NT * pieces - 1) / (kRun * NT * pieces);
}

// A row's shares: a piece for each thread while that makes up to 512 workgroups;
// else two at least, and up to 1024 workgroups (16 rows of 131072 logits: 10.7 us
// with two pieces, 11.7 with one, 11.2 with four; 128 rows: 18.3 with 1024
// workgroups, 20.2 with 512, 19.9 with 2048).
int32_t shares_of(int32_t n, int32_t vocab)
{
    const int64_t one = shares_with(vocab, 1), two = shares_with(vocab, 2);
    if (n * one <= 512)
        return (int32_t)one;
    const int64_t want = 1024 / n;
    return (int32_t)(want < 1 ? 1 : want < two ? want : two);
}

constexpr int64_t kShareBytes = (NT + 4) * sizeof(float);

template <typename T>
hipError_t launch_typed(const kvr_ctx *c, const LogprobArgs &a, hipStream_t s)
{
    const hipError_t e = launch(c, KVR_KERNEL_LOGPROB, part_kernel<T>,
                                dim3((unsigned)((int64_t)a.c.n * a.shares)), dim3(NT), 0, s, a);
    if (e != hipSuccess)
        return e;
    // (512 rows of 32000 logits, 2 shares: 20.0 us with 256 threads a row, 21.2 with
    // 1024; 128 rows of 131072, 8 shares: 18.6, 17.6; one row, 64 shares: 26, 9.8)
    if (a.shares <= 4)
        return launch(c, KVR_KERNEL_LOGPROB, row_kernel<T, 256, 4>, dim3((unsigned)a.c.n),
                      dim3(256), 0, s, a);
    return launch(c, KVR_KERNEL_LOGPROB, row_kernel<T, 1024, 16>, dim3((unsigned)a.c.n), dim3(1024),
                  0, s, a);
}

}  // namespace

// Of exactly that call, and the largest over calls of fewer rows or logits.
int64_t logprob_workspace(int32_t n, int32_t vocab)
{
    return n * (int64_t)shares_of(n, vocab) * kShareBytes;
}

int64_t logprob_workspace_bound(int32_t n, int32_t vocab)
{
    const int64_t most = shares_with(vocab, 1) * n;
    const int64_t many = n > 1024 ? n : 1024;
    return (most < many ? most : many) * kShareBytes;
}

hipError_t launch_logprob(const kvr_ctx *c, const kvr_logprob_call &p, hipStream_t s)
{
    LogprobArgs a{};
    a.c = p;
    a.pieces = (int32_t)(((int64_t)p.vocab + kRun - 1) / kRun);
    a.shares = shares_of(p.n, p.vocab);
    a.per = (a.pieces + a.shares * NT - 1) / (a.shares * NT) * NT;
    a.wide = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
             p.logits_stride * value_bytes(p.value_type) % 16 == 0;
    a.parts = static_cast<float *>(p.workspace);
    a.tops = a.parts + (int64_t)p.n * a.shares * 4;
    if (p.value_type == KVR_VALUE_F32)
        return launch_typed<float>(c, a, s);
    if (p.value_type == KVR_VALUE_BF16)
        return launch_typed<__bf16>(c, a, s);
    return launch_typed<_Float16>(c, a, s);
}

}  // namespace kvr
