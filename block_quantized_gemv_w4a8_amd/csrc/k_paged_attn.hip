// k_paged_attn.hip -- attention over a paged cache with causal order, an
// optional sliding window and the first keys that stay visible.
//
// One pass over the keys with the running maximum m and sum l of a softmax:
// for each group of keys, m' = max(m, max x), o and l are scaled by
// exp(m - m'), and exp(x - m') v and exp(x - m') are added.
#include "qgemv_layer.h"

namespace qgemv {

struct AttnDev {
    const void *q, *k, *v;
    void* out;
    float* lse;
    const int32_t *q_start, *kv_len, *table;
    int64_t ldq, ldo, ldt, page_stride, token_stride, head_stride;
    int T, q_heads, heads, G, D, B, max_q, n_pages, page_size, window, sinks;
    float scale;
};

// One query row over its keys, by one wave: 64 keys at a time, a key to a
// lane for the scores, then the values with the row's dimensions over the
// lanes.  No key that the row does not see is read.
template <typename T, typename TO>
__global__ __launch_bounds__(256) void k_attn_row(const AttnDev a) {
    const int lane = threadIdx.x & 63;
    const int64_t rows = (int64_t)a.max_q * a.q_heads;
    const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    const int b = blockIdx.y;
    if (r >= rows) return;
    const int i = (int)(r / a.q_heads), hq = (int)(r % a.q_heads), h = hq / a.G;
    const int s0 = min(max(a.q_start[b], 0), a.T);
    const int s1 = min(max(a.q_start[b + 1], s0), a.T);
    if (i >= s1 - s0) return;
    const int64_t p = (int64_t)a.kv_len[b] - (s1 - s0) + i;
    const int64_t top = min(p + 1, a.ldt * a.page_size);           // keys before it
    const int64_t z = a.window > 0 ? max(p - a.window + 1, (int64_t)0) : 0;
    const int64_t sink = min((int64_t)a.sinks, z);
    const T* q = (const T*)a.q + (int64_t)(s0 + i) * a.ldq + (int64_t)hq * a.D;
    const T* k = (const T*)a.k + h * a.head_stride;
    const T* v = (const T*)a.v + h * a.head_stride;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const int64_t n = sink + max(top - z, (int64_t)0);
    for (int64_t g = 0; g < n; g += 64) {
        const int64_t idx = g + lane;
        const int64_t j = idx < sink ? idx : z + idx - sink;
        int64_t at = -1;
        if (idx < n && j < top) {
            const int page = a.table[b * a.ldt + j / a.page_size];
            if (page >= 0 && page < a.n_pages)
                at = page * a.page_stride + (j % a.page_size) * a.token_stride;
        }
        float x = -INFINITY;
        if (at >= 0) {
            x = 0.f;
            for (int d = 0; d < a.D; d += 8) {
                float kf[8], qf[8];
                load8(k + at + d, kf);
                load8(q + d, qf);
#pragma unroll
                for (int e = 0; e < 8; e++) x = fmaf(qf[e], kf[e], x);
            }
            x *= a.scale;
        }
        float mg = x;
        for (int w = 32; w; w >>= 1) mg = fmaxf(mg, __shfl_xor(mg, w));
        const float mn = fmaxf(m, mg);
        if (mn == -INFINITY) continue;
        const float fix = expf(m - mn), pr = at >= 0 ? expf(x - mn) : 0.f;
        float sum = pr;
        for (int w = 32; w; w >>= 1) sum += __shfl_xor(sum, w);
        l = l * fix + sum;
        m = mn;
#pragma unroll
        for (int c = 0; c < 4; c++) o[c] *= fix;
        for (int t = 0; t < 64; t++) {
            const int64_t tat = __shfl((long long)at, t);
            const float tp = __shfl(pr, t);
            if (tat < 0) continue;
#pragma unroll
            for (int c = 0; c < 4; c++)
                if (lane + 64 * c < a.D) o[c] = fmaf(tp, (float)v[tat + lane + 64 * c], o[c]);
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    TO* out = (TO*)a.out + (int64_t)(s0 + i) * a.ldo + (int64_t)hq * a.D;
#pragma unroll
    for (int c = 0; c < 4; c++)
        if (lane + 64 * c < a.D) out[lane + 64 * c] = (TO)(o[c] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t)(s0 + i) * a.q_heads + hq] = l != 0.f ? m + logf(l) : -INFINITY;
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t st) {
    AttnDev d{};
    d.q = a.q; d.k = a.c.k; d.v = a.c.v; d.out = a.out; d.lse = a.lse;
    d.q_start = a.q_start; d.kv_len = a.kv_len; d.table = a.table;
    d.ldq = a.ldq; d.ldo = a.ldo; d.ldt = a.ldt;
    d.page_stride = a.c.page_stride; d.token_stride = a.c.token_stride;
    d.head_stride = a.c.head_stride;
    d.T = a.T; d.q_heads = a.q_heads; d.heads = a.c.heads; d.G = a.q_heads / a.c.heads;
    d.D = a.c.head_dim; d.B = a.B; d.max_q = a.max_q; d.n_pages = a.c.n_pages;
    d.page_size = a.c.page_size; d.window = a.window; d.sinks = a.sinks; d.scale = a.scale;
    const dim3 grid((unsigned)(((int64_t)a.max_q * a.q_heads + 3) / 4), (unsigned)a.B);
    with_type16(a.c.type, [&](auto t) {
        with_type(a.out_type, [&](auto to) {
            launch_kernel(k_attn_row<decltype(t), decltype(to)>, grid, dim3(256), 0, st, d);
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
