// k_rope_append.hip -- rotary positions of new q and k rows, and k and v into
// their slots of a paged cache.
//
// With a = pos * inv_freq[i], (x_i, x_j) -> (x_i cos a - x_j sin a, x_j cos a +
// x_i sin a).  The angle is formed in 64 bits and reduced to a fraction of a
// turn there, because a 32-bit product near 10^6 is off by up to 2^-5 of a
// radian, which leaves 7 or 8 bits of the turn; sine and cosine are then fp32.  They are the same
// for every head of a token, so a workgroup, which has one token or a part of
// it, forms the rot_dim / 2 pairs once, in LDS.  Everything else is memory
// traffic: each value is read once from memory and written once, 8 at a time.

#include <algorithm>

#include "qgemv_layer.h"

namespace qgemv {

constexpr int RWG = 256;

// How the rotated part is walked, a chunk of 8 values a lane.  Halves: the chunk
// of the partners is fetched beside it (it is on its way for another lane: a
// lane with both chunks would fetch each once, but store parts of lines, and
// took 61 us where this takes 43 for 8192 tokens of 48 heads of 128, half of it
// rotated: 4.7 TB/s, of 5.3 that a copy reaches).  Pairs: the partners are in the
// chunk.  Single handles any even rot_dim and fetches each partner by itself (the
// same tokens with 122 of 128 rotated 75 us, 2.7 TB/s; 40 of 80 in halves 50 us,
// 2.5 TB/s).
enum RopeWalk { kHalves, kPairs, kSingle };

struct RopeDev {
    const void *q, *k, *v;
    void *q_out, *kc, *vc;
    const int32_t* pos;
    const int64_t* slots;
    const float* inv_freq;
    int64_t ldq, ldk, ldv, ldqo, page_stride, token_stride, head_stride, n_slots;
    int64_t first;  // the launch's first token
    int q_heads, heads, D, rot, page_size, style;
    int items;  // chunks of a token
};

template <typename TI, typename TO, RopeWalk WALK>
__global__ __launch_bounds__(RWG) void k_rope_append(const RopeDev a) {
    __shared__ float2 cs[QGEMV_HEAD_DIM_MAX / 2];
    const int half = a.rot / 2;
    const int64_t tok = a.first + blockIdx.x;
    const int64_t slot = a.slots[tok];
    for (int f = threadIdx.x; f < half; f += RWG) {
        const double turns = (double)a.pos[tok] * (double)a.inv_freq[f] * 0.15915494309189535;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[f] = make_float2(c, s);
    }
    const bool stored = slot >= 0 && slot < a.n_slots;
    int64_t place = 0;   // element offset of the slot
    if (stored) {
        const uint32_t page = (uint64_t)slot / (uint32_t)a.page_size;
        place = page * a.page_stride + (slot - (int64_t)page * a.page_size) * a.token_stride;
    }
    __syncthreads();
    const int per = a.D / 8, qk = a.q_heads + a.heads;
    for (int it = blockIdx.y * RWG + threadIdx.x; it < a.items; it += gridDim.y * RWG) {
        const int hh = it / per, e0 = 8 * (it - hh * per);   // heads of q, then of k, then of v
        const bool is_q = hh < a.q_heads, is_v = hh >= qk;
        if (!is_q && !stored) continue;
        const int h = is_q ? hh : is_v ? hh - qk : hh - a.q_heads;
        const TI* src = (is_q ? (const TI*)a.q + tok * a.ldq
                              : is_v ? (const TI*)a.v + tok * a.ldv : (const TI*)a.k + tok * a.ldk) +
                        (int64_t)h * a.D;
        TO* dst = is_q ? (TO*)a.q_out + tok * a.ldqo + (int64_t)h * a.D
                       : (TO*)(is_v ? a.vc : a.kc) + place + h * a.head_stride;
        float x[8];
        load8(src + e0, x);
        if (!is_v && e0 < a.rot) {
            if constexpr (WALK == kHalves) {
                const bool first = e0 < half;
                float y[8];
                load8(src + (first ? e0 + half : e0 - half), y);
                const float2* w = cs + (first ? e0 : e0 - half);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    x[i] = first ? x[i] * w[i].x - y[i] * w[i].y : x[i] * w[i].x + y[i] * w[i].y;
            } else if constexpr (WALK == kPairs) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 w = cs[(e0 + i) / 2];
                    const float u = x[i];
                    x[i] = u * w.x - x[i + 1] * w.y;
                    x[i + 1] = x[i + 1] * w.x + u * w.y;
                }
            } else {
                const bool pairs = a.style == QGEMV_ROPE_PAIRS;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int e = e0 + i;
                    if (e >= a.rot) continue;
                    const bool first = pairs ? !(e & 1) : e < half;
                    const float2 w = cs[pairs ? e / 2 : (first ? e : e - half)];
                    const float u = (float)src[pairs ? e ^ 1 : (first ? e + half : e - half)];
                    x[i] = first ? x[i] * w.x - u * w.y : x[i] * w.x + u * w.y;
                }
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
    d.q_heads = a.q_heads; d.heads = a.c.heads; d.D = a.c.head_dim; d.rot = a.rot_dim;
    d.page_size = a.c.page_size; d.style = a.style;
    const RopeWalk walk = a.style == QGEMV_ROPE_HALVES ? (a.rot_dim % 16 == 0 ? kHalves : kSingle)
                                                       : (a.rot_dim % 8 == 0 ? kPairs : kSingle);
    d.items = (d.q_heads + 2 * d.heads) * (d.D / 8);
    // few tokens: all of a token's chunks at once; many: one workgroup a token,
    // which forms its angles once
    const int rows = (d.items + RWG - 1) / RWG;
    // (a launch has fewer than 2^32 threads; what is past them would be left out
    // without an error)
    constexpr int kTokens = 1 << 23;
    with_type(a.in_type, [&](auto ti) {
        with_type16(a.c.type, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            for (d.first = 0; d.first < a.T; d.first += kTokens) {
                const dim3 grid((unsigned)std::min<int64_t>(a.T - d.first, kTokens),
                                (unsigned)(a.T <= 512 ? rows : 1));
                if (walk == kHalves)
                    launch_kernel(k_rope_append<TI, TO, kHalves>, grid, dim3(RWG), 0, st, d);
                else if (walk == kPairs)
                    launch_kernel(k_rope_append<TI, TO, kPairs>, grid, dim3(RWG), 0, st, d);
                else
                    launch_kernel(k_rope_append<TI, TO, kSingle>, grid, dim3(RWG), 0, st, d);
            }
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
