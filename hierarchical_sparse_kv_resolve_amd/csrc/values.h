// Reading and writing runs of values of the types that calls take.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvr.h"

namespace kvr {

constexpr int64_t value_bytes(int32_t value_type) { return value_type == KVR_VALUE_F32 ? 4 : 2; }

constexpr bool value_type_ok(int32_t t)
{
    return t == KVR_VALUE_BF16 || t == KVR_VALUE_F16 || t == KVR_VALUE_F32;
}

// N consecutive values as 32-bit floats; `wide`: the address is aligned to 16
// bytes (or to all of the values, if they are fewer).
template <int N, typename T>
__device__ __forceinline__ void load_run(const T *p, bool wide, float (&x)[N])
{
    constexpr int M = N * sizeof(T) > 16 ? 16 / sizeof(T) : N;  // values of one load
    typedef T vec __attribute__((ext_vector_type(M)));
    if (wide) {
#pragma unroll
        for (int i = 0; i < N; i += M) {
            const vec v = *reinterpret_cast<const vec *>(p + i);
#pragma unroll
            for (int j = 0; j < M; ++j)
                x[i + j] = (float)v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = (float)p[i];
    }
}

template <int N, typename T>
__device__ __forceinline__ void store_run(T *p, bool wide, const float (&x)[N])
{
    constexpr int M = N * sizeof(T) > 16 ? 16 / sizeof(T) : N;
    typedef T vec __attribute__((ext_vector_type(M)));
    if (wide) {
#pragma unroll
        for (int i = 0; i < N; i += M) {
            vec v;
#pragma unroll
            for (int j = 0; j < M; ++j)
                v[j] = (T)x[i + j];
            *reinterpret_cast<vec *>(p + i) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            p[i] = (T)x[i];
    }
}

}  // namespace kvr
