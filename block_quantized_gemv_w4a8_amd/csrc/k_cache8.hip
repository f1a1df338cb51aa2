// k_cache8.hip -- the 8-bit paged cache as it is written (rotary positions of new
// q and k rows, k and v quantised into their slots) and as plain rows again.
//
// Append: with a = pos * inv_freq[i], (x_i, x_j) -> (x_i cos a - x_j sin a, x_j
// cos a + x_i sin a); then for each row of k and v d = max|y| / 127 and codes
// round(y / d).  A code changes where y / d passes a border, so y is one number
// whatever the order of operations: sine and cosine are 64-bit ones rounded to
// fp32, products of two fp32 numbers are exact in 64 bits, and their sum is rounded
// once to fp32.  (The 64-bit part is two conversions, a product and an fma a value
// at the rate of fp32, about a tenth of what the memory's way takes.)  The
// angles are formed once a workgroup, in LDS; a row's lanes find its maximum among
// themselves.
#include <algorithm>

#include "qgemv_rows.h"

namespace qgemv {

constexpr int RWG = 256;

// How the rotated part is walked, a chunk of 8 values a lane: partners a chunk
// further on (rot_dim a multiple of 16), in the chunk, or each by itself.
enum RopeWalk { kHalves, kPairs, kSingle };

struct Rope8Dev {
    const void *q, *k, *v;
    void *q_out;
    int8_t *kc, *vc;
    float *ks, *vs;
    const int32_t* pos;
    const int64_t* slots;
    const float* inv_freq;
    int64_t ldq, ldk, ldv, ldqo, page_stride, token_stride, head_stride, n_slots;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    int64_t first;  // the launch's first token
    int q_heads, heads, D, rot, page_size, style;
};

// x c - y s, or with -s x c + y s, formed in 64 bits and rounded once.
__device__ __forceinline__ float turned(float x, float c, float y, float s) {
    return (float)fma((double)x, (double)c, -((double)y * (double)s));
}

// LPR lanes a row (a power of two, at least D / 8).  Bound by memory and by the way
// to the angles, which stand before a workgroup's work: 8192 tokens of 48 heads of 128,
// half of each rotated, 48.6 us, 3.8 TB/s of 5.3 that a copy reaches (with a row's loads
// ahead of the row before it 54); all of each 53, by pairs 41.  kSingle reads partners one by
// one: 122 of 128 values rotated 71 us, by pairs 83.
template <typename TI, typename TQ, RopeWalk WALK, int LPR>
__global__ __launch_bounds__(RWG) void k_rope_append8(const Rope8Dev a) {
    __shared__ float2 cs[QGEMV_HEAD_DIM_MAX / 2];
    const int half = a.rot / 2;
    const int64_t tok = a.first + blockIdx.x;
    const int64_t slot = a.slots[tok];
    for (int f = threadIdx.x; f < half; f += RWG) {
        double s, c;
        sincos((double)a.pos[tok] * (double)a.inv_freq[f], &s, &c);
        cs[f] = make_float2((float)c, (float)s);
    }
    const bool stored = slot >= 0 && slot < a.n_slots;
    int64_t place = 0, scale_place = 0;   // offsets of the slot
    if (stored) {
        const uint32_t page = (uint64_t)slot / (uint32_t)a.page_size;
        const int64_t in = slot - (int64_t)page * a.page_size;
        place = page * a.page_stride + in * a.token_stride;
        scale_place = page * a.scale_page_stride + in * a.scale_token_stride;
    }
    __syncthreads();
    constexpr int RPP = RWG / LPR;
    const int rows = a.q_heads + 2 * a.heads, qk = a.q_heads + a.heads;
    const int lane = threadIdx.x % LPR, e0 = 8 * lane;
    const bool there = e0 < a.D;
    for (int hh = blockIdx.y * RPP + threadIdx.x / LPR; hh < rows; hh += gridDim.y * RPP) {
        const bool is_q = hh < a.q_heads, is_v = hh >= qk;   // heads of q, then of k, then of v
        if (!is_q && !stored) continue;
        const int h = is_q ? hh : is_v ? hh - qk : hh - a.q_heads;
        const TI* src = (is_q ? (const TI*)a.q + tok * a.ldq
                              : is_v ? (const TI*)a.v + tok * a.ldv : (const TI*)a.k + tok * a.ldk) +
                        (int64_t)h * a.D;
        float x[8] = {};
        if (there) load8(src + e0, x);
        if (!is_v && e0 < a.rot) {
            if constexpr (WALK == kHalves) {
                const bool first = e0 < half;
                float y[8];
                load8(src + (first ? e0 + half : e0 - half), y);
                const float2* w = cs + (first ? e0 : e0 - half);
#pragma unroll
                for (int i = 0; i < 8; i++) x[i] = turned(x[i], w[i].x, y[i], first ? w[i].y : -w[i].y);
            } else if constexpr (WALK == kPairs) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 w = cs[(e0 + i) / 2];
                    const float u = x[i];
                    x[i] = turned(u, w.x, x[i + 1], w.y);
                    x[i + 1] = turned(x[i + 1], w.x, u, -w.y);
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
                    x[i] = turned(x[i], w.x, u, first ? w.y : -w.y);
                }
            }
        }
        if (is_q) {
            if (there) store8((TQ*)a.q_out + tok * a.ldqo + (int64_t)h * a.D + e0, x);
            continue;
        }
        float top = top8(x);
#pragma unroll
        for (int w = LPR / 2; w; w >>= 1) top = fmaxf(top, __shfl_xor(top, w));
        const float d = row_scale(top);
        if (there)
            *reinterpret_cast<uint2*>((is_v ? a.vc : a.kc) + place + h * a.head_stride + e0) = codes8(x, d);
        if (lane == 0) (is_v ? a.vs : a.ks)[scale_place + h * a.scale_head_stride] = d;
    }
}

hipError_t launch_rope_append_q8(const Rope8Args& a, hipStream_t st) {
    Rope8Dev d{};
    d.q = a.q; d.k = a.k; d.v = a.v; d.q_out = a.q_out;
    d.kc = (int8_t*)a.c.k; d.vc = (int8_t*)a.c.v; d.ks = a.c.k_scale; d.vs = a.c.v_scale;
    d.pos = a.pos; d.slots = a.slots; d.inv_freq = a.inv_freq;
    d.ldq = a.ldq; d.ldk = a.ldk; d.ldv = a.ldv; d.ldqo = a.ldqo;
    d.page_stride = a.c.page_stride; d.token_stride = a.c.token_stride;
    d.head_stride = a.c.head_stride;
    d.scale_page_stride = a.c.scale_page_stride; d.scale_token_stride = a.c.scale_token_stride;
    d.scale_head_stride = a.c.scale_head_stride;
    d.n_slots = (int64_t)a.c.n_pages * a.c.page_size;
    d.q_heads = a.q_heads; d.heads = a.c.heads; d.D = a.c.head_dim; d.rot = a.rot_dim;
    d.page_size = a.c.page_size; d.style = a.style;
    const RopeWalk walk = a.style == QGEMV_ROPE_HALVES ? (a.rot_dim % 16 == 0 ? kHalves : kSingle)
                                                       : (a.rot_dim % 8 == 0 ? kPairs : kSingle);
    // (a launch has fewer than 2^32 threads; what is past them would be left out
    // without an error)
    constexpr int kTokens = 1 << 23;
    with_type(a.in_type, [&](auto ti) {
        with_type16(a.q_heads > 0 ? a.q_type : QGEMV_TYPE_BF16, [&](auto tq) {
            using TI = decltype(ti);
            using TQ = decltype(tq);
            auto go = [&](auto kernel, int lpr) {
                // few tokens: all of a token's rows at once; many: one workgroup a token,
                // which forms its angles once (48 heads of 128 in three parts: 1 token 3.5 us and
                // 4.8, 256 5.3 and 6.4, 512 6.9 and 7.4, 768 9.3 and 9.1, 2048 17.2 and 16.2, 8192 65 and 52)
                const int64_t rows = (int64_t)d.q_heads + 2 * d.heads;
                const int64_t parts = (rows * lpr + RWG - 1) / RWG;
                for (d.first = 0; d.first < a.T; d.first += kTokens)
                    launch_kernel(kernel, dim3((unsigned)std::min<int64_t>(a.T - d.first, kTokens),
                                               (unsigned)(a.T <= 512 ? parts : 1)),
                                  dim3(RWG), 0, st, d);
            };
            auto walks = [&](auto lpr) {
                constexpr int LPR = decltype(lpr)::value;
                if (walk == kHalves) go(k_rope_append8<TI, TQ, kHalves, LPR>, LPR);
                else if (walk == kPairs) go(k_rope_append8<TI, TQ, kPairs, LPR>, LPR);
                else go(k_rope_append8<TI, TQ, kSingle, LPR>, LPR);
            };
            if (d.D <= 64) walks(std::integral_constant<int, 8>{});
            else if (d.D <= 128) walks(std::integral_constant<int, 16>{});
            else walks(std::integral_constant<int, 32>{});
        });
    });
    return hipGetLastError();
}

struct Read8Dev {
    const int8_t *kc, *vc;
    const float *ks, *vs;
    const int64_t* slots;
    void *k_out, *v_out;
    int64_t ldk, ldv, page_stride, token_stride, head_stride, n_slots;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    uint32_t items, per;   // chunks of the launch, and of a token
    int D, page_size;
};

// A store of 16 bytes a thread for k and one for v.  Bound by memory: 40001 slots of 8
// heads of 128 to bf16 51.5 us, 4.8 TB/s of 5.3 that a copy reaches.
template <typename TO>
__global__ __launch_bounds__(256) void k_cache_read8(const Read8Dev a) {
    constexpr int VPL = 16 / sizeof(TO);
    const uint32_t it = blockIdx.x * 256u + threadIdx.x;
    if (it >= a.items) return;
    const uint32_t t = it / a.per, c = VPL * (it - t * a.per), h = c / (uint32_t)a.D, e = c - h * a.D;
    const int64_t slot = a.slots[t];
    const bool there = slot >= 0 && slot < a.n_slots;
    int64_t place = 0, scale_place = 0;
    if (there) {
        const uint32_t page = (uint64_t)slot / (uint32_t)a.page_size;
        const int64_t in = slot - (int64_t)page * a.page_size;
        place = page * a.page_stride + in * a.token_stride + h * a.head_stride + e;
        scale_place = page * a.scale_page_stride + in * a.scale_token_stride + h * a.scale_head_stride;
    }
    auto put = [&](const int8_t* codes, const float* scales, void* out, int64_t ld) {
        if (!out) return;
        alignas(8) int8_t q[VPL] = {};
        float d = 0.f;
        if (there) {
            __builtin_memcpy(q, __builtin_assume_aligned(codes + place, VPL), VPL);
            d = scales[scale_place];
        }
        alignas(16) TO f[VPL];
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            float x = there ? (float)q[i] * d : 0.f;
            asm volatile("" : "+v"(x));   // (a value is an fp32 number, whatever it is then rounded to)
            f[i] = (TO)x;
        }
        *reinterpret_cast<uint4*>((TO*)out + t * ld + c) = *reinterpret_cast<const uint4*>(f);
    };
    put(a.kc, a.ks, a.k_out, a.ldk);
    put(a.vc, a.vs, a.v_out, a.ldv);
}

hipError_t launch_cache_read_q8(const Read8Args& a, hipStream_t st) {
    Read8Dev d{};
    d.kc = (const int8_t*)a.c.k; d.vc = (const int8_t*)a.c.v; d.ks = a.c.k_scale; d.vs = a.c.v_scale;
    d.ldk = a.ldk; d.ldv = a.ldv;
    d.page_stride = a.c.page_stride; d.token_stride = a.c.token_stride;
    d.head_stride = a.c.head_stride;
    d.scale_page_stride = a.c.scale_page_stride; d.scale_token_stride = a.c.scale_token_stride;
    d.scale_head_stride = a.c.scale_head_stride;
    d.n_slots = (int64_t)a.c.n_pages * a.c.page_size;
    d.D = a.c.head_dim; d.page_size = a.c.page_size;
    with_type(a.out_type, [&](auto to) {
        using TO = decltype(to);
        d.per = (uint32_t)((int64_t)a.c.heads * d.D * sizeof(TO) / 16);
        // (pieces, so that a launch's chunks are counted in 32 bits)
        const int64_t piece = std::max<int64_t>(1, (1 << 30) / d.per);
        for (int64_t t = 0; t < a.T; t += piece) {
            const int64_t n = std::min(a.T - t, piece);
            d.items = (uint32_t)(n * d.per);
            d.slots = a.slots + t;
            d.k_out = a.k_out ? (TO*)a.k_out + t * a.ldk : nullptr;
            d.v_out = a.v_out ? (TO*)a.v_out + t * a.ldv : nullptr;
            launch_kernel(k_cache_read8<TO>, dim3((d.items + 255) / 256), dim3(256), 0, st, d);
        }
    });
    return hipGetLastError();
}

}  // namespace qgemv
