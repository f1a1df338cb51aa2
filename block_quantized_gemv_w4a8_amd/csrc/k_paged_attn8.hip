// k_paged_attn8.hip -- attention over a paged cache of int8 codes with one scale a
// row, with causal order, an optional sliding window and the first keys that stay
// visible.
//
// With codes ck, cv and scales sk, sv: x_j = scale sk_j (q . ck_j), m their
// largest, w_j = exp(x_j - m), out = sum w_j sv_j cv_j / sum w_j.
#include "qgemv_attn.h"

namespace qgemv {

struct Attn8Dev : AttnDev {     // (strides of codes in bytes)
    const float *ks, *vs;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
};

__device__ __forceinline__ int64_t scale_offset(const Attn8Dev& a, int page, int j) {
    const int in = a.page_shift >= 0 ? j & (a.page_size - 1) : j % a.page_size;
    return page * a.scale_page_stride + in * a.scale_token_stride;
}

// One row over one part of its keys, by one wave: a key to a lane for the
// scores, then the dimensions over the lanes.  It touches no key that the row
// does not see, and stands in for the matrix path where something of an unseen
// key that is not finite (0 * inf) has spoilt the row's sum.
template <typename T, int KT>
__device__ void attn8_row(const Attn8Dev& a, const Span& s, const int32_t* table, int i, int hq,
                          float c2, float (&o)[4], float& m, float& l) {
    const int lane = threadIdx.x & 63;
    const int h = hq / a.G, p = s.place(i), z = window_start(a, p);
    const T* q = (const T*)a.q + (int64_t)(s.s0 + i) * a.ldq + (int64_t)hq * a.D;
    const int8_t* k = (const int8_t*)a.k + h * a.head_stride;
    const int8_t* v = (const int8_t*)a.v + h * a.head_stride;
    m = -INFINITY;
    l = 0.f;
    for (int c = 0; c < 4; c++) o[c] = 0.f;
    for (int t = s.t0; t < s.t1; t++) {
        const int j = tile_of(s, t) * KT + lane;
        int64_t at = -1, scale_at = 0;
        if (lane < KT && j <= p && (j >= z || j < a.sinks)) {
            const int page = page_of(a, table, j, s.limit);
            if (page >= 0 && page < a.n_pages) {
                at = key_offset(a, page, j);
                scale_at = scale_offset(a, page, j) + h * a.scale_head_stride;
            }
        }
        float x = -INFINITY, sv = 0.f;
        if (at >= 0) {
            x = 0.f;
            for (int d = 0; d < a.D; d += 8) {
                float qf[8];
                load8(q + d, qf);
                const uint2 c = *reinterpret_cast<const uint2*>(k + at + d);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    x = fmaf(qf[e], (float)(int8_t)((e < 4 ? c.x : c.y) >> (8 * (e % 4))), x);
            }
            x = x * a.ks[scale_at] * c2;
            sv = a.vs[scale_at];
        }
        float mt = x;
        for (int w = 32; w; w >>= 1) mt = fmaxf(mt, __shfl_xor(mt, w));
        const float mn = fmaxf(m, mt);
        // (a NaN among the scores leaves the maximum as it is, and has to count)
        if (mn == -INFINITY && !__any(x != x)) continue;
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float fix = exp2f(m - mu), pr = at >= 0 ? exp2f(x - mu) : 0.f;
        float sum = pr;
        for (int w = 32; w; w >>= 1) sum += __shfl_xor(sum, w);
        l = l * fix + sum;
        m = mn;
        // (o, like l, takes a tile at once, so that a long flat tail is not lost from it)
        float add[4] = {0.f, 0.f, 0.f, 0.f};
        for (int u = 0; u < KT; u++) {
            const int64_t tat = __shfl((long long)at, u);
            const float tp = __shfl(pr * sv, u);
            if (tat < 0) continue;
            for (int c = 0; c < 4; c++)
                if (lane + 64 * c < a.D) add[c] = fmaf(tp, (float)v[tat + lane + 64 * c], add[c]);
        }
        for (int c = 0; c < 4; c++) o[c] = o[c] * fix + add[c];
    }
}

// A wave a row.
template <typename T, typename TO>
__global__ __launch_bounds__(64) void k_attn8_rows(const Attn8Dev a) {
    const int b = blockIdx.y;
    for (int r = blockIdx.x; r < a.max_q * a.q_heads; r += gridDim.x) {
        const int i = r / a.q_heads, hq = r - i * a.q_heads;
        Span s;
        if (!make_span<64, 1>(a, b, i * a.G, 0, s)) return;
        float o[4], m, l;
        attn8_row<T, 64>(a, s, a.table + b * a.ldt, i, hq, a.scale * 1.4426950408889634f, o, m, l);
        put_row<TO>(a, s, 0, i, hq, o, m, l);
    }
}

hipError_t launch_paged_attn_q8(const Attn8Args& a, hipStream_t st) {
    Attn8Dev d{};
    d.q = a.q; d.k = a.c.k; d.v = a.c.v; d.ks = a.c.k_scale; d.vs = a.c.v_scale;
    d.out = a.out; d.lse = a.lse;
    d.q_start = a.q_start; d.kv_len = a.kv_len; d.table = a.table;
    d.ldq = a.ldq; d.ldo = a.ldo; d.ldt = a.ldt;
    d.page_stride = a.c.page_stride; d.token_stride = a.c.token_stride;
    d.head_stride = a.c.head_stride;
    d.scale_page_stride = a.c.scale_page_stride; d.scale_token_stride = a.c.scale_token_stride;
    d.scale_head_stride = a.c.scale_head_stride;
    d.T = a.T; d.q_heads = a.q_heads; d.heads = a.c.heads; d.G = a.q_heads / a.c.heads;
    d.D = a.c.head_dim; d.B = a.B; d.max_q = a.max_q; d.n_pages = a.c.n_pages;
    d.page_size = a.c.page_size; d.window = a.window; d.sinks = a.sinks; d.scale = a.scale;
    d.page_shift = (a.c.page_size & (a.c.page_size - 1)) == 0 ? __builtin_ctz(a.c.page_size) : -1;
    d.splits = d.split_tiles = 1;
    with_type16(a.q_type, [&](auto t) {
        with_type(a.out_type, [&](auto to) {
            launch_kernel(k_attn8_rows<decltype(t), decltype(to)>,
                          dim3((unsigned)std::min(d.max_q * d.q_heads, 1 << 20), (unsigned)d.B), dim3(64), 0, st, d);
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
