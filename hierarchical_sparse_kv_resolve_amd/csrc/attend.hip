// Attention of new tokens over resolved rows.
#include "block.h"
#include "kvr_internal.h"
#include "rowformat.h"

namespace kvr {
namespace {

constexpr int NT = 256;

struct AttendArgs {
    Shape sh;
    const LayerPtrs *layers;
    kvr_attend_call c;
};

// Address of entry j of request entry i, or null when it is left out.
__device__ __forceinline__ const uint8_t *row_address(const AttendArgs &a, const LayerPtrs &lp, int i,
                                                      int r, int64_t j, bool &bad)
{
    bad = false;
    const int64_t e = (int64_t)i * a.c.stride + j;
    const uint32_t w = a.c.loc ? a.c.loc[e] : 0;
    if (w == KVR_LOC_INVALID)
        return nullptr;
    if (a.c.rows)
        return static_cast<const uint8_t *>(a.c.rows) + e * a.sh.R;
    const uint32_t place = w >> kPlaceShift, idx = w & kIndexMask;
    if (place == KVR_PLACE_TAIL && idx < (uint32_t)a.sh.T)
        return lp.tail + ((int64_t)r * a.sh.T + idx) * a.sh.R;
    if (place == KVR_PLACE_PAGE && (int64_t)idx < a.sh.pool_rows)
        return lp.pool + (int64_t)idx * a.sh.R;
    if (place == KVR_PLACE_HOT && (idx & kSlotMask) < (uint32_t)a.sh.B)
        return lp.hot + ((int64_t)r * a.sh.B + (idx & kSlotMask)) * a.sh.R;
    bad = true;
    return nullptr;
}

template <int FMT>
__device__ float key_value(const uint8_t *row, int d_v, int d)
{
    typedef typename Elem<FMT>::type E;
    if constexpr (FMT == KVR_ROW_FP8) {
        if (d >= d_v)
            return (float)reinterpret_cast<const E *>(row + d_v + scale_bytes(d_v))[d - d_v];
        const float sc = reinterpret_cast<const float *>(row + d_v)[d / kScaleGroup];
        return __builtin_amdgcn_cvt_f32_fp8((int)row[d], 0) * sc;
    } else {
        return (float)reinterpret_cast<const E *>(row)[d];
    }
}

// One workgroup per (entry, query, head), one row per thread and step.
template <int FMT>
__global__ __launch_bounds__(NT) void attend_kernel(AttendArgs a)
{
    typedef typename Elem<FMT>::type E;
    __shared__ float sQ[576], sP[NT], sRed[NT];
    __shared__ const uint8_t *sRow[NT];
    const int64_t b = blockIdx.x;
    const int h = (int)(b % a.c.heads), qi = (int)(b / a.c.heads % a.c.nq),
              i = (int)(b / a.c.heads / a.c.nq);
    const int r = a.c.req_ids ? a.c.req_ids[i] : i;
    const bool badr = r < 0 || r >= a.sh.n_req;
    int cnt = a.c.count ? a.c.count[i] : a.c.stride;
    cnt = cnt < 0 ? 0 : (cnt > a.c.stride ? a.c.stride : cnt);
    const int D = a.c.d_v + a.c.d_rope;
    const E *q = static_cast<const E *>(a.c.q) + i * a.c.q_stride_entry +
                 qi * a.c.q_stride_query + h * a.c.q_stride_head;
    for (int d = threadIdx.x; d < D; d += NT)
        sQ[d] = (float)q[d];
    const int n = badr ? 0 : (a.c.map ? a.c.k : cnt);
    if (badr && threadIdx.x == 0 && a.c.status)
        a.c.status[i] = KVR_E_ARG;
    LayerPtrs lp{};
    if (!a.c.rows && n > 0)
        lp = a.layers[a.c.layer];
    float m = -__builtin_inff(), l = 0.f, o[2] = {0.f, 0.f};
    for (int j0 = 0; j0 < n; j0 += NT) {
        __syncthreads();
        const int j = j0 + threadIdx.x;
        const uint8_t *row = nullptr;
        if (j < n) {
            const int64_t e = a.c.map ? a.c.map[((int64_t)i * a.c.nq + qi) * a.c.k + j] : j;
            bool bad = false;
            if (e >= 0 && e < cnt)
                row = row_address(a, lp, i, r, e, bad);
            if (bad && a.c.status)
                a.c.status[i] = KVR_E_RANGE;
        }
        float s = -__builtin_inff();
        if (row) {
            s = 0.f;
            for (int d = 0; d < D; ++d)
                s += sQ[d] * key_value<FMT>(row, a.c.d_v, d);
            s *= a.c.scale;
        }
        sRow[threadIdx.x] = row;
        sRed[threadIdx.x] = s;
        __syncthreads();
        float mt = m;
        for (int t = 0; t < NT; ++t)
            mt = (mt > sRed[t] || mt != mt) ? mt : sRed[t];
        const float base = mt == -__builtin_inff() ? 0.f : mt;
        const float alpha = expf(m - base);
        sP[threadIdx.x] = row ? expf(s - base) : 0.f;
        __syncthreads();
        l *= alpha;
        o[0] *= alpha;
        o[1] *= alpha;
        for (int t = 0; t < NT; ++t) {
            if (!sRow[t])
                continue;
            l += sP[t];
            for (int u = 0; u < 2; ++u) {
                const int d = u * NT + threadIdx.x;
                if (d < a.c.d_v)
                    o[u] += sP[t] * key_value<FMT>(sRow[t], a.c.d_v, d);
            }
        }
        m = mt;
    }
    E *out = static_cast<E *>(a.c.out) + b * a.c.d_v;
    for (int u = 0; u < 2; ++u) {
        const int d = u * NT + threadIdx.x;
        if (d < a.c.d_v)
            out[d] = (E)(m == -__builtin_inff() ? 0.f : o[u] / l);
    }
    if (threadIdx.x == 0 && a.c.lse)
        a.c.lse[b] = m == -__builtin_inff() ? m : m + logf(l);
}

}  // namespace

AttendPlan attend_plan(int32_t, int32_t, int32_t, int32_t, int32_t, bool)
{
    return AttendPlan{1, 1, 1, 0};
}

int64_t attend_workspace_bound(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_attend(const kvr_ctx *c, const kvr_attend_call &call, const AttendPlan &,
                         hipStream_t s)
{
    AttendArgs a{c->shape, c->layers_d, call};
    const dim3 grid((unsigned)((int64_t)call.n * call.nq * call.heads));
    if (call.format == KVR_ROW_FP8)
        return launch(c, KVR_KERNEL_ATTEND, attend_kernel<KVR_ROW_FP8>, grid, dim3(NT), 0, s, a);
    if (call.format == KVR_ROW_BF16)
        return launch(c, KVR_KERNEL_ATTEND, attend_kernel<KVR_ROW_BF16>, grid, dim3(NT), 0, s, a);
    return launch(c, KVR_KERNEL_ATTEND, attend_kernel<KVR_ROW_F16>, grid, dim3(NT), 0, s, a);
}

}  // namespace kvr
