// attention_simple.cuh -- the paged attention in its simplest form: one warp
// per query row, one key at a time, softmax by a running maximum and sum.
#pragma once

#include "attention_common.cuh"

namespace kvq {

struct RowState {
    float m, l, acc[4];
    __device__ __forceinline__ void init() {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = 0.0f;
    }
    template <int E>
    __device__ __forceinline__ void key(float s, const float (&v)[E]) {
        const float mn = fmaxf(m, s);
        if (mn == -INFINITY) return;
        const float c = exp2f(m - mn), p = exp2f(s - mn);
        l = __fmaf_rn(l, c, p);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = __fmaf_rn(p, v[i], acc[i] * c);
        m = mn;
    }
};

template <int T, int C, int D>
__global__ void __launch_bounds__(128) shared_simple_kernel(const SharedArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (w >= a.B * a.Nq) return;
    const int b = w / a.Nq, h = w - b * a.Nq, kh = h / a.G;
    const int32_t n = own_length(a, b);
    if (n < 0) return;
    float q[E], sk[E], sv[E], ok[E], ov[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = kh * D + lane + 32 * e;
        q[e] = att_load<T>(a.q.base, (int64_t)b * a.q.tok + h * a.q.head + lane + 32 * e);
        sk[e] = C == ATT_I8 ? a.scale_k[c] : 1.0f;
        sv[e] = C == ATT_I8 ? a.scale_v[c] : 1.0f;
        ok[e] = C == ATT_I8 && a.offset_k ? a.offset_k[c] : 0.0f;
        ov[e] = C == ATT_I8 && a.offset_v ? a.offset_v[c] : 0.0f;
    }
    RowState r;
    r.init();
    for (int32_t t = 0; t < a.prefix_len + n; ++t) {
        int32_t at;
        const int32_t page = t < a.prefix_len ? page_of(a, a.prefix_table, t, &at)
                                              : page_of(a, a.table + (int64_t)b * a.table_stride, t - a.prefix_len, &at);
        if (page < 0) continue;
        const int64_t o = ((int64_t)at * a.Nkv + kh) * D + lane;
        const uint8_t* kp = a.k_cache + page * a.k_page;
        const uint8_t* vp = a.v_cache + page * a.v_page;
        float d = 0.0f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            d = __fmaf_rn(q[e], (att_load<C>(kp, o + 32 * e) - ok[e]) * sk[e], d);
            v[e] = (att_load<C>(vp, o + 32 * e) - ov[e]) * sv[e];
        }
        r.key(warp_sum(d) * (a.scale * ATT_LOG2E), v);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        att_store<T>(a.out.base, (int64_t)b * a.out.tok + h * a.out.head + lane + 32 * e,
                     r.l > 0.0f ? __fdiv_rn(r.acc[e], r.l) : 0.0f);
    if (a.lse && lane == 0) a.lse[(int64_t)b * a.Nq + h] = (r.m + log2f(r.l)) * ATT_LN2;
}

}  // namespace kvq
