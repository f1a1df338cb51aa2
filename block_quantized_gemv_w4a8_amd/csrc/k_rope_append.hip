// k_rope_append.hip -- rotary positions of new q and k rows, and k and v into
// their slots of a paged cache.
//
// With a = pos * inv_freq[i], (x_i, x_j) -> (x_i cos a - x_j sin a, x_j cos a +
// x_i sin a).  The angle is formed in 64 bits and reduced to a fraction of a
// turn there, because a position of 10^6 leaves a 32-bit product only ~4
// correct bits of the turn; sine and cosine are then fp32.  They are the same
// for every head of a token, so a workgroup forms the rot_dim / 2 pairs of
// its tokens once, in LDS.  Everything else is memory traffic: each value is
// read once and written once, 8 at a time.
#include "qgemv_layer.h"

namespace qgemv {

constexpr int RWG = 256;

// How the rotated part is walked.  Halves and Pairs move whole chunks of 8
// values (a pair of chunks for Halves); Single handles any even rot_dim and
// fetches each partner by itself.
enum RopeWalk { kHalves, kPairs, kSingle };

struct RopeDev {
    const void *q, *k, *v;
    void *q_out, *kc, *vc;
    const int32_t* pos;
    const int64_t* slots;
    const float* inv_freq;
    int64_t ldq, ldk, ldv, ldqo, page_stride, token_stride, head_stride, n_slots;
    int T, q_heads, heads, D, rot, page_size, style;
    int per_head, items;  // work items of a q or k head, and of a token
};

template <typename TI, typename TO, RopeWalk WALK>
__global__ __launch_bounds__(RWG) void k_rope_append(const RopeDev a, int tokens) {
    __shared__ float2 cs[8][QGEMV_HEAD_DIM_MAX / 2];
    const int half = a.rot / 2;
    const int t0 = blockIdx.x * tokens;
    const int nt = min(tokens, a.T - t0);
    for (int i = threadIdx.x; i < nt * half; i += RWG) {
        const int t = i / half, f = i - t * half;
        const double turns = (double)a.pos[t0 + t] * (double)a.inv_freq[f] * 0.15915494309189535;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[t][f] = make_float2(c, s);
    }
    __syncthreads();
    const int qk = a.q_heads + a.heads;
    for (int it = blockIdx.y * RWG + threadIdx.x; it < nt * a.items; it += gridDim.y * RWG) {
        const int t = it / a.items;
        const int r = it - t * a.items;
        const int64_t tok = t0 + t;
        const bool is_v = r >= qk * a.per_head;
        const int per = is_v ? a.D / 8 : a.per_head;
        const int rr = is_v ? r - qk * a.per_head : r;
        const int hh = rr / per, ch = rr - hh * per;
        const bool is_q = !is_v && hh < a.q_heads;
        const int h = is_q || is_v ? hh : hh - a.q_heads;
        const TI* src;
        TO* dst;
        if (is_q) {
            src = (const TI*)a.q + tok * a.ldq + (int64_t)h * a.D;
            dst = (TO*)a.q_out + tok * a.ldqo + (int64_t)h * a.D;
        } else {
            const int64_t slot = a.slots[tok];
            if (slot < 0 || slot >= a.n_slots) continue;
            const int64_t page = slot / a.page_size;
            const int64_t at = page * a.page_stride + (slot - page * a.page_size) * a.token_stride +
                               h * a.head_stride;
            src = (const TI*)(is_v ? a.v : a.k) + tok * (is_v ? a.ldv : a.ldk) + (int64_t)h * a.D;
            dst = (TO*)(is_v ? a.vc : a.kc) + at;
        }
        float x[8];
        if (!is_v && WALK == kHalves && 8 * ch < half) {
            float y[8], xo[8], yo[8];
            load8(src + 8 * ch, x);
            load8(src + half + 8 * ch, y);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float2 w = cs[t][8 * ch + i];
                xo[i] = x[i] * w.x - y[i] * w.y;
                yo[i] = y[i] * w.x + x[i] * w.y;
            }
            store8(dst + 8 * ch, xo);
            store8(dst + half + 8 * ch, yo);
            continue;
        }
        // a chunk of its own: the copied tail of a head, v, a chunk of whole
        // pairs, or one whose partners are fetched singly
        const int e0 = 8 * (!is_v && WALK == kHalves ? ch + half / 8 : ch);
        load8(src + e0, x);
        if (!is_v && WALK == kPairs && e0 < a.rot) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 w = cs[t][(e0 + i) / 2];
                const float u = x[i];
                x[i] = u * w.x - x[i + 1] * w.y;
                x[i + 1] = x[i + 1] * w.x + u * w.y;
            }
        }
        if (!is_v && WALK == kSingle) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int e = e0 + i;
                if (e >= a.rot) continue;
                const bool pairs = a.style == QGEMV_ROPE_PAIRS;
                const bool first = pairs ? !(e & 1) : e < half;
                const int f = pairs ? e / 2 : (first ? e : e - half);
                const int o = pairs ? e ^ 1 : (first ? e + half : e - half);
                const float2 w = cs[t][f];
                const float u = (float)src[o];
                x[i] = first ? x[i] * w.x - u * w.y : x[i] * w.x + u * w.y;
            }
        }
        store8(dst + e0, x);
    }
}

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
    RopeDev d{};
    d.q = a.q; d.k = a.k; d.v = a.v; d.q_out = a.q_out; d.kc = a.c.k; d.vc = a.c.v;
    d.pos = a.pos; d.slots = a.slots; d.inv_freq = a.inv_freq;
    d.ldq = a.ldq; d.ldk = a.ldk; d.ldv = a.ldv; d.ldqo = a.ldqo;
    d.page_stride = a.c.page_stride; d.token_stride = a.c.token_stride;
    d.head_stride = a.c.head_stride;
    d.n_slots = (int64_t)a.c.n_pages * a.c.page_size;
    d.T = a.T; d.q_heads = a.q_heads; d.heads = a.c.heads; d.D = a.c.head_dim; d.rot = a.rot_dim;
    d.page_size = a.c.page_size; d.style = a.style;
    const RopeWalk walk = a.style == QGEMV_ROPE_HALVES ? (a.rot_dim % 16 == 0 ? kHalves : kSingle)
                                                       : (a.rot_dim % 8 == 0 ? kPairs : kSingle);
    d.per_head = d.D / 8 - (walk == kHalves ? d.rot / 16 : 0);
    d.items = (d.q_heads + d.heads) * d.per_head + d.heads * (d.D / 8);
    const int tokens = 1;
    const dim3 grid((unsigned)((a.T + tokens - 1) / tokens), 1);
    with_type(a.in_type, [&](auto ti) {
        with_type16(a.c.type, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            if (walk == kHalves)
                launch_kernel(k_rope_append<TI, TO, kHalves>, grid, dim3(RWG), 0, st, d, tokens);
            else if (walk == kPairs)
                launch_kernel(k_rope_append<TI, TO, kPairs>, grid, dim3(RWG), 0, st, d, tokens);
            else
                launch_kernel(k_rope_append<TI, TO, kSingle>, grid, dim3(RWG), 0, st, d, tokens);
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
