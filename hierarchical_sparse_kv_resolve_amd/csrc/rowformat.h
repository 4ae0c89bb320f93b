// The row formats that kvr_pack_rows writes and kvr_attend_rows reads: the
// latent of a token (d_v values), then its rope part (d_rope values).
//   16-bit   d_v + d_rope values of bf16 or fp16
//   fp8      d_v e4m3 codes, one 32-bit scale per 128 of them (the scale area
//            rounded up to 16 bytes), d_rope values of bf16
#pragma once

#include <stdint.h>

#include "block.h"
#include "kvr.h"

namespace kvr {

constexpr int kScaleGroup = 128;    // values per scale
constexpr float kE4m3Max = 448.0f;  // largest finite e4m3 value

__host__ __device__ constexpr int scale_bytes(int d_v)
{
    return (d_v / kScaleGroup * 4 + 15) / 16 * 16;
}

constexpr bool row_dims_ok(int32_t d_v, int32_t d_rope)
{
    return (d_v == 256 || d_v == 512) && (d_rope == 0 || d_rope == 64);
}

constexpr int32_t row_bytes_of(int32_t format, int32_t d_v, int32_t d_rope)
{
    return format == KVR_ROW_FP8 ? d_v + scale_bytes(d_v) + 2 * d_rope : 2 * (d_v + d_rope);
}

// The 16-bit type of a format (an fp8 row's rope part and the queries and
// outputs that go with it are bf16).
template <int FMT>
struct Elem {
    typedef __bf16 type;
};
template <>
struct Elem<KVR_ROW_F16> {
    typedef _Float16 type;
};

// Sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum_f32(float x)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        x += __shfl_xor(x, m);
    return x;
}

// Maximum over aligned groups of LANES lanes; NaN wins.
template <int LANES>
__device__ __forceinline__ float group_max_f32(float x)
{
#pragma unroll
    for (int m = LANES / 2; m >= 1; m >>= 1) {
        const float y = __shfl_xor(x, m);
        x = (x > y || x != x) ? x : y;
    }
    return x;
}

// Four values rounded to e4m3 (nearest, ties to even), first in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

}  // namespace kvr
