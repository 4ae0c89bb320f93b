// Rows of new tokens in the cache's format: the RMS norm of each token's
// latent, then 16-bit values, or e4m3 codes with one scale for each group of
// 128 values, then the token's rope part in 16 bits.  ("Adaptive DHiSparse",
// section "How it works": the resolver moves rows as opaque bytes; this is
// the kernel that writes them and kvr_attend_rows the one that reads them.)
//
//   x = latent * 1/sqrt(mean(latent^2) + eps) * weight      (32-bit sums)
//   fp8: scale = max|x| / 448 of its group (1 for a group of zeros),
//        code = e4m3(x / scale), so that a group's largest code is 448
//
// One wave owns a row: a lane holds d_v / 64 consecutive values, so a scale
// group of 128 is 16 lanes (d_v 512) or 32 lanes (d_v 256) and its maximum is
// a few lane exchanges.  One pass over the data, the next row's loads issued
// before a row is worked on, bound by HBM: 131072 rows of 512 + 64 bf16 values
// to fp8 (237 MB) in 47 us, 5.0 TB/s, to fp16 (302 MB) in 55 us, 5.5 TB/s.
// (With inputs left in the cache by the call before, a division for each value
// took 54 us, bound by vector instructions, where the reciprocal took 43, and
// without the early loads it took 59.)
#include "block.h"
#include "kvr_internal.h"
#include "rowformat.h"

namespace kvr {
namespace {

constexpr int NT = 256;
constexpr float kTinyScale = 1e-36f;  // 1 / scale is finite above it

struct PackArgs {
    int64_t n;
    const void *latent, *rope;
    int64_t latent_stride, rope_stride;  // elements
    const float *weight;                 // null: no norm
    float eps;
    uint8_t *rows;
    int32_t row_bytes;
    int32_t d_rope;
};

template <int N>
struct Raw16 {
    uint16_t v[N];
};

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__bf16>(__bf16 x) { return (float)x; }
template <>
__device__ __forceinline__ float to_f32<_Float16>(_Float16 x) { return (float)x; }

// N consecutive values; `wide`: the address is aligned to all of them (8 to 32
// bytes).
template <int N, typename T>
__device__ __forceinline__ void load_values(const T *p, bool wide, float (&x)[N])
{
    if (wide) {
        typedef T vec __attribute__((ext_vector_type(N)));
        const vec v = *reinterpret_cast<const vec *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = to_f32<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = to_f32<T>(p[i]);
    }
}

// Row n of the call by one wave.
template <int FMT, int DV, typename T>
__global__ __launch_bounds__(NT) void pack_kernel(PackArgs a, bool wide)
{
    constexpr int N = DV / 64;
    typedef typename Elem<FMT>::type E;
    const int lane = lane_id();
    const int64_t waves = (int64_t)gridDim.x * (NT / 64);
    float w[N];
    if (a.weight)
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = a.weight[lane * N + i];
    // a row's values are loaded while the row before is worked on
    float x[N], nx[N], rope = 0.f, nrope = 0.f;
    auto load = [&](int64_t row) {
        if (row >= a.n)
            return;
        load_values<N>(static_cast<const T *>(a.latent) + row * a.latent_stride + lane * N, wide, nx);
        if (lane < a.d_rope)
            nrope = to_f32<T>(static_cast<const T *>(a.rope)[row * a.rope_stride + lane]);
    };
    int64_t row = (int64_t)blockIdx.x * (NT / 64) + wave_id();
    load(row);
    for (; row < a.n; row += waves) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = nx[i];
        rope = nrope;
        load(row + waves);
        if (a.weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                ss = fmaf(x[i], x[i], ss);
            ss = wave_sum_f32(ss);
            const float inv = 1.0f / sqrtf(ss * (1.0f / DV) + a.eps);
#pragma unroll
            for (int i = 0; i < N; ++i)
                x[i] = x[i] * inv * w[i];
        }
        uint8_t *out = a.rows + row * a.row_bytes;
        if constexpr (FMT == KVR_ROW_FP8) {
            float top = 0.f;
            bool nan = false;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                top = fmaxf(top, fabsf(x[i]));
                nan |= x[i] != x[i];
            }
            top = nan ? __builtin_nanf("") : top;
            top = group_max_f32<kScaleGroup / N>(top);
            float scale = top / kE4m3Max;
            scale = scale == 0.f ? 1.f : scale;
            // by the reciprocal (two roundings instead of one, both far below a
            // code's), except where that would overflow.  A subnormal scale is a
            // whole number of 2^-149 and may be up to a third too small: its
            // quotients are held to the largest code (a NaN stays one).
            const float inv = 1.f / scale;
            if (__any(scale < kTinyScale)) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float y = x[i] / scale;
                    x[i] = y > kE4m3Max ? kE4m3Max : y < -kE4m3Max ? -kE4m3Max : y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    x[i] *= inv;
            }
            uint32_t code[N / 4];
#pragma unroll
            for (int i = 0; i < N; i += 4)
                code[i / 4] = pack_e4m3(x[i], x[i + 1], x[i + 2], x[i + 3]);
            typedef uint32_t codes __attribute__((ext_vector_type(N / 4)));
            codes cv;
            __builtin_memcpy(&cv, code, sizeof cv);
            *reinterpret_cast<codes *>(out + lane * N) = cv;
            constexpr int kLanes = kScaleGroup / N;  // lanes of one group
            constexpr int kScaleWords = scale_bytes(DV) / 4;
            // every 4-byte word of the scale area is written (unused ones 0)
            const float sv = __shfl(scale, (lane % (DV / kScaleGroup)) * kLanes);
            if (lane < kScaleWords)
                *reinterpret_cast<float *>(out + DV + 4 * lane) =
                    lane < DV / kScaleGroup ? sv : 0.f;
            if (lane < a.d_rope)
                *reinterpret_cast<E *>(out + DV + scale_bytes(DV) + 2 * lane) = (E)rope;
        } else {
            typedef E vec __attribute__((ext_vector_type(N)));
            vec v;
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = (E)x[i];
            *reinterpret_cast<vec *>(out + lane * N * 2) = v;
            if (lane < a.d_rope)
                *reinterpret_cast<E *>(out + DV * 2 + 2 * lane) = (E)rope;
        }
    }
}

template <int FMT, int DV>
hipError_t launch_typed(const kvr_ctx *c, int32_t src, const PackArgs &a, bool wide, dim3 grid,
                        hipStream_t s)
{
    if (src == KVR_VALUE_F32)
        return launch(c, KVR_KERNEL_PACK, pack_kernel<FMT, DV, float>, grid, dim3(NT), 0, s, a, wide);
    if (src == KVR_VALUE_BF16)
        return launch(c, KVR_KERNEL_PACK, pack_kernel<FMT, DV, __bf16>, grid, dim3(NT), 0, s, a, wide);
    return launch(c, KVR_KERNEL_PACK, pack_kernel<FMT, DV, _Float16>, grid, dim3(NT), 0, s, a, wide);
}

template <int FMT>
hipError_t launch_format(const kvr_ctx *c, int32_t d_v, int32_t src, const PackArgs &a, bool wide,
                         dim3 grid, hipStream_t s)
{
    return d_v == 512 ? launch_typed<FMT, 512>(c, src, a, wide, grid, s)
                      : launch_typed<FMT, 256>(c, src, a, wide, grid, s);
}

}  // namespace

hipError_t launch_pack(const kvr_ctx *c, const kvr_pack_call &p, hipStream_t s)
{
    PackArgs a{};
    a.n = p.n;
    a.latent = p.latent;
    a.rope = p.rope;
    a.latent_stride = p.latent_stride;
    a.rope_stride = p.rope_stride;
    a.weight = p.weight;
    a.eps = p.eps;
    a.rows = static_cast<uint8_t *>(p.rows);
    a.row_bytes = c->shape.R;
    a.d_rope = p.d_rope;
    // a lane's values are loaded in one piece when each row's start allows it
    const int64_t e = p.value_type == KVR_VALUE_F32 ? 4 : 2;
    const int64_t piece = e * (p.d_v / 64);
    const bool wide = reinterpret_cast<uintptr_t>(p.latent) % piece == 0 &&
                      (p.latent_stride * e) % piece == 0;
    const int64_t blocks = (p.n + NT / 64 - 1) / (NT / 64);
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (p.format == KVR_ROW_FP8)
        return launch_format<KVR_ROW_FP8>(c, p.d_v, p.value_type, a, wide, grid, s);
    if (p.format == KVR_ROW_BF16)
        return launch_format<KVR_ROW_BF16>(c, p.d_v, p.value_type, a, wide, grid, s);
    return launch_format<KVR_ROW_F16>(c, p.d_v, p.value_type, a, wide, grid, s);
}

}  // namespace kvr
