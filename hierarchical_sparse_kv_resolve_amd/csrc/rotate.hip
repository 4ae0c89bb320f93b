// Rotary positions of queries and keys: pair i of a head's rotated part, at
// position p, turns by a = 2 pi p f_i:
//   u' = magnitude (u cos a - v sin a),  v' = magnitude (v cos a + u sin a).
//
// p f_i is taken in 64 bits and loses its whole turns there (32 bits would leave
// an error of p 2^-24 turns); sines and cosines are 32-bit.  A workgroup first
// puts those of its tokens into LDS, once for all heads (a 64-bit product, a sine and
// a cosine a pair would cost more than the turn itself), then walks the heads, 16
// bytes a thread where addresses allow.  Bound by HBM, every value being read and
// written once: 32768 tokens of 20 heads of 128 bf16 values 60 us, 336 MB at 5.6 TB/s
// (partly from the Infinity Cache); 64 tokens of 16 heads of 576 4.9 us, a launch and
// two dependent loads.
#include "block.h"
#include "kvr_internal.h"
#include "values.h"

namespace kvr {
namespace {

constexpr int NT = 256;
constexpr int kTable = 1024;  // pairs in LDS

struct Part {
    kvr_rotate_part p;
    bool wide;      // 16 bytes at a time
    int32_t turned; // units of a head's rotated part
    int32_t units;  // and those copied
};

struct RotateArgs {
    Part part[2];
    const int32_t *positions;
    const double *frequencies;
    int32_t n, d_rot, tokens;  // tokens of a workgroup
    int32_t splits;            // workgroups that share them
    float magnitude, sign;
};

// A unit of a head: U pairs that are turned (HALF: U values of either half, else
// 2 U values side by side), or as many values that are copied (one, with U = 1).
template <typename T, bool HALF, int U>
__device__ __forceinline__ void rotate_unit(const kvr_rotate_part &p, const float2 *table,
                                            int64_t token, int head, int unit, int turned,
                                            int d_rot)
{
    constexpr int V = HALF ? U : 2 * U;  // consecutive values
    const T *x = static_cast<const T *>(p.x) + token * p.x_stride_token + head * p.x_stride_head;
    T *out = static_cast<T *>(p.out) + token * p.out_stride_token + head * p.out_stride_head;
    constexpr bool wide = U > 1;
    if (unit >= turned) {
        constexpr int C = wide ? V : 1;
        typedef T vec __attribute__((ext_vector_type(C)));
        int d = (unit - turned) * C;
        d += d >= p.at ? d_rot : 0;
        *reinterpret_cast<vec *>(out + d) = *reinterpret_cast<const vec *>(x + d);
        return;
    }
    const float2 *cs = table + unit * U;
    const int d = p.at + unit * V;
    if constexpr (HALF) {
        float u[U], v[U];
        load_run<U>(x + d, wide, u);
        load_run<U>(x + d + d_rot / 2, wide, v);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float2 c = cs[k];
            const float a = u[k];
            u[k] = a * c.x - v[k] * c.y;
            v[k] = v[k] * c.x + a * c.y;
        }
        store_run<U>(out + d, wide, u);
        store_run<U>(out + d + d_rot / 2, wide, v);
    } else {
        float y[2 * U];
        load_run<2 * U>(x + d, wide, y);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float2 c = cs[k];
            const float a = y[2 * k];
            y[2 * k] = a * c.x - y[2 * k + 1] * c.y;
            y[2 * k + 1] = y[2 * k + 1] * c.x + a * c.y;
        }
        store_run<2 * U>(out + d, wide, y);
    }
}

template <typename T, bool HALF>
__global__ __launch_bounds__(NT) void rotate_kernel(RotateArgs a)
{
    constexpr int kPiece = 16 / sizeof(T);
    constexpr int U = HALF ? kPiece : kPiece / 2;  // pairs of a 16-byte unit
    __shared__ float2 sTable[kTable];
    const int pairs = a.d_rot / 2;
    const int64_t first = (int64_t)(blockIdx.x / a.splits) * a.tokens;
    const int split = blockIdx.x % a.splits;
    const int tokens = (int)(a.n - first < a.tokens ? a.n - first : a.tokens);
    for (int q = threadIdx.x; q < tokens * pairs; q += NT) {
        const int t = q / pairs, i = q - t * pairs;
        const double turns = (double)a.positions[first + t] * a.frequencies[i];
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        sTable[q] = make_float2(c * a.magnitude, s * a.magnitude * a.sign);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const Part &part = a.part[w];
        const int per = part.p.heads * part.units;  // units of a token
        for (int64_t q = (int64_t)split * NT + threadIdx.x; q < (int64_t)tokens * per;
             q += (int64_t)a.splits * NT) {
            const int t = (int)(q / per), in = (int)(q - (int64_t)t * per);
            const int head = in / part.units, unit = in - head * part.units;
            if (part.wide)
                rotate_unit<T, HALF, U>(part.p, sTable + t * pairs, first + t, head, unit,
                                        part.turned, a.d_rot);
            else
                rotate_unit<T, HALF, 1>(part.p, sTable + t * pairs, first + t, head, unit,
                                        part.turned, a.d_rot);
        }
    }
}

template <typename T>
hipError_t launch_layout(const kvr_ctx *c, bool half, const RotateArgs &a, dim3 grid, hipStream_t s)
{
    return half ? launch(c, KVR_KERNEL_ROTATE, rotate_kernel<T, true>, grid, dim3(NT), 0, s, a)
                : launch(c, KVR_KERNEL_ROTATE, rotate_kernel<T, false>, grid, dim3(NT), 0, s, a);
}

}  // namespace

hipError_t launch_rotate(const kvr_ctx *c, const kvr_rotate_call &r, hipStream_t s)
{
    RotateArgs a{};
    a.positions = r.positions;
    a.frequencies = r.frequencies;
    a.n = r.n;
    a.d_rot = r.d_rot;
    a.magnitude = r.magnitude;
    a.sign = r.inverse ? -1.f : 1.f;
    const bool half = r.layout == KVR_ROPE_HALF;
    const int64_t piece = 16 / value_bytes(r.value_type);
    int64_t units = 0;  // of a token
    for (int w = 0; w < 2; ++w) {
        Part &p = a.part[w];
        p.p = w ? r.key : r.query;
        if (p.p.heads == 0)
            continue;
        const bool in_place = p.p.x == p.p.out;
        const int32_t rest = in_place ? 0 : p.p.d_head - r.d_rot;
        p.wide = (reinterpret_cast<uintptr_t>(p.p.x) | reinterpret_cast<uintptr_t>(p.p.out)) % 16 == 0 &&
                 (p.p.x_stride_token | p.p.x_stride_head | p.p.out_stride_token |
                  p.p.out_stride_head | p.p.at | rest | (half ? r.d_rot / 2 : r.d_rot)) % piece == 0;
        const int32_t values = p.wide ? (int32_t)piece : 1;
        p.turned = half ? r.d_rot / 2 / values : r.d_rot / (p.wide ? values : 2);
        p.units = p.turned + rest / values;
        units += (int64_t)p.p.heads * p.units;
    }
    if (units == 0)
        return hipSuccess;
    const int pairs = r.d_rot / 2;
    // Tokens of a workgroup: until each thread has a unit, no more than the table
    // holds, and fewer where there are not 1024 workgroups.  32768 tokens of 40 heads
    // of 128 (320 units a token) 115 us with one token, 130 with 8; of 20 heads 61
    // with 2, 64 with 1 and 65 with 8; 4096 tokens of 16 heads of 576, 64 of them
    // turned, 38 with 1, 42 with 8.
    int64_t tokens = 1;
    while (tokens * units < NT && 2 * tokens <= kTable / pairs && r.n / (2 * tokens) >= 1024)
        tokens *= 2;
    a.tokens = (int32_t)tokens;
    const int64_t groups = (r.n + tokens - 1) / tokens;
    // Workgroups share tokens that are two rounds or more for one, up to 1024 of them
    // and a round each (1160 units: 64 tokens in a workgroup each 5.9 us, in 5 3.7, 192
    // tokens 6.2 and 4.4, 400 8.4 and 7.2; 320 units: 256 tokens 3.8, in two 4.6).
    int64_t splits = 1024 / groups;
    const int64_t most = tokens * units < 2 * NT ? 1 : (tokens * units + NT - 1) / NT;
    splits = splits < most ? splits : most;
    a.splits = (int32_t)(splits < 1 ? 1 : splits);
    const dim3 grid((unsigned)(groups * a.splits));
    if (r.value_type == KVR_VALUE_F32)
        return launch_layout<float>(c, half, a, grid, s);
    if (r.value_type == KVR_VALUE_BF16)
        return launch_layout<__bf16>(c, half, a, grid, s);
    return launch_layout<_Float16>(c, half, a, grid, s);
}

}  // namespace kvr
