// qgemv_attn.h -- what the attention kernels over a paged cache share, whatever the
// cache's values are held in: the sequences' spans of keys, the rows' results, and
// the split of keys over workgroups with the launch that joins it.
#pragma once

#include <algorithm>
#include <type_traits>

#include "qgemv_layer.h"

namespace qgemv {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(1))) const void gmem;
typedef __attribute__((address_space(3))) void lmem;
typedef __attribute__((address_space(3))) s16x4 lmem4;

struct AttnDev {
    const void *q, *k, *v;
    void* out;
    float *lse, *part_o, *part_ml;
    const int32_t *q_start, *kv_len, *table;
    int64_t ldq, ldo, ldt, page_stride, token_stride, head_stride;
    int T, q_heads, heads, G, D, B, max_q, n_pages, page_size, page_shift, window, sinks;
    int row_tiles, splits, split_tiles;
    float scale;
    bool runs;      // 16 keys from a multiple of 16 share a page, and their offsets in it are small
};

// The queries of a sequence and the keys that a block of its rows sees, as a
// list of tiles: those of the sinks, then those from the window's start.
struct Span {
    int s0, n, kv;          // first query, queries, keys
    int i0, i1;             // queries of the block
    int limit;              // keys that are there and that the table can hold
    int sink_tiles, win_tile, tiles;
    int t0, t1, parts;      // this part of the list, and how many parts it has

    __device__ __forceinline__ int place(int i) const { return kv - n + i; }
};

__device__ __forceinline__ int window_start(const AttnDev& a, int p) {
    return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

template <int KT, int ROWS>
__device__ __forceinline__ bool make_span(const AttnDev& a, int b, int row_tile, int part, Span& s) {
    s.s0 = min(max(a.q_start[b], 0), a.T);
    s.n = min(max(a.q_start[b + 1], s.s0), a.T) - s.s0;
    s.kv = max(a.kv_len[b], 0);
    s.i0 = row_tile * ROWS / a.G;
    const int last = min(s.n, a.max_q) - 1;
    if (s.i0 > last) return false;
    s.i1 = min((row_tile * ROWS + ROWS - 1) / a.G, last);
    // (kept below 2^31 with room for a tile)
    s.limit = (int)min(min(a.ldt * a.page_size, (int64_t)0x7fffff00), (int64_t)s.kv);
    const int top = min(s.place(s.i1) + 1, s.limit);
    const int z = window_start(a, s.place(s.i0));
    const int sink = max(min(min(a.sinks, z), top), 0);
    s.sink_tiles = (sink + KT - 1) / KT;
    s.win_tile = max(z / KT, s.sink_tiles);
    s.tiles = s.sink_tiles + (top > 0 ? max((top + KT - 1) / KT - s.win_tile, 0) : 0);
    const int each = max(a.split_tiles, (s.tiles + a.splits - 1) / a.splits);
    s.parts = max(1, (s.tiles + each - 1) / each);
    s.t0 = min(part * each, s.tiles);
    s.t1 = min(s.t0 + each, s.tiles);
    return part < s.parts;
}
__device__ __forceinline__ int tile_of(const Span& s, int t) {
    return t < s.sink_tiles ? t : s.win_tile + t - s.sink_tiles;
}

// The page of key j, -1 where it has none; and the key's element offset.
__device__ __forceinline__ int page_of(const AttnDev& a, const int32_t* table, int j, int limit) {
    if (j >= limit) return -1;
    const int c = a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size;
    return table[c];
}
__device__ __forceinline__ int64_t key_offset(const AttnDev& a, int page, int j) {
    const int in = a.page_shift >= 0 ? j & (a.page_size - 1) : j % a.page_size;
    return page * a.page_stride + in * a.token_stride;
}

// m is in units of log2; 1 / l of a row that saw nothing is 0.
__device__ __forceinline__ float row_inverse(float l) { return l != 0.f ? 1.f / l : 0.f; }
__device__ __forceinline__ float row_lse(float m, float l) {
    return l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// A row's result from `o` in the layout of attn_row.
template <typename TO>
__device__ void put_row(const AttnDev& a, const Span& s, int part, int i, int hq,
                        const float (&o)[4], float m, float l) {
    const int lane = threadIdx.x & 63;
    const int64_t t = s.s0 + i, row = t * a.q_heads + hq;
    if (s.parts > 1) {
        const int64_t at = row * a.splits + part;
        for (int c = 0; c < 4; c++)
            if (lane + 64 * c < a.D) a.part_o[at * a.D + lane + 64 * c] = o[c];
        if (lane == 0) {
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
        return;
    }
    const float inv = row_inverse(l);
    TO* out = (TO*)a.out + t * a.ldo + (int64_t)hq * a.D;
    for (int c = 0; c < 4; c++)
        if (lane + 64 * c < a.D) out[lane + 64 * c] = (TO)(o[c] * inv);
    if (a.lse && lane == 0) a.lse[row] = row_lse(m, l);
}

#define QGEMV_WAIT(...) asm volatile("s_waitcnt " __VA_ARGS__ ::: "memory")
#define QGEMV_BARRIER()                    \
    do {                                   \
        __builtin_amdgcn_s_barrier();      \
        asm volatile("" ::: "memory");     \
    } while (0)

// The larger of a lane's value and of the one 32 lanes on.
__device__ __forceinline__ float max_halves(float x) {
    const int own = __builtin_bit_cast(int, x);
    const auto r = __builtin_amdgcn_permlane32_swap(own, own, false, false);
    const int lo = r[0], hi = r[1];   // (a bit cast of r[1] itself is compiled as one of r[0])
    return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// Joins the parts of the rows whose keys were split: LANES lanes a row, four
// dimensions each, eight parts in flight (18 rows of 32 heads in five parts: 4.4
// us, where a wave a row and part after part took 11.7).
template <typename TO, int KT, int ROWS, int LANES>
__global__ __launch_bounds__(256) void k_attn_join(const AttnDev a) {
    const int r = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;  // query and head of the sequence
    const int d = 4 * (threadIdx.x % LANES), b = blockIdx.y;
    const int i = r / a.q_heads, hq = r - i * a.q_heads, h = hq / a.G;
    if (i >= a.max_q || d >= a.D) return;
    // the place of the row's parts needs its sequence's start only, and the first
    // parts are asked for before it is known how many there are
    const int s0 = min(max(a.q_start[b], 0), a.T);
    const int64_t tok = s0 + i, row = tok * a.q_heads + hq;
    const float* ml = a.part_ml + 2 * row * a.splits;
    const float* po = a.part_o + row * a.splits * a.D + d;
    constexpr int AHEAD = 8;
    float m[AHEAD], l[AHEAD];
    f32x4v v[AHEAD];
#pragma unroll
    for (int w = 0; w < AHEAD; w++) {
        if (tok >= a.T || w >= a.splits) continue;
        m[w] = ml[2 * w];
        l[w] = ml[2 * w + 1];
        v[w] = *reinterpret_cast<const f32x4v*>(po + (int64_t)w * a.D);
    }
    Span s;
    const int row_tile = (i * a.G + hq - h * a.G) / ROWS;
    if (!make_span<KT, ROWS>(a, b, row_tile, 0, s) || i >= s.n || s.parts == 1) return;
    float top = -INFINITY, sum = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < AHEAD; w++)
        if (w < s.parts) top = fmaxf(top, m[w]);
    for (int w = AHEAD; w < s.parts; w++) top = fmaxf(top, ml[2 * w]);
    auto join = [&](float mw, float lw, const f32x4v& vw) {
        const float fix = mw == top ? 1.f : exp2f(mw - top);
        sum += lw * fix;
#pragma unroll
        for (int c = 0; c < 4; c++) f[c] += vw[c] * fix;
    };
#pragma unroll
    for (int w = 0; w < AHEAD; w++)
        if (w < s.parts) join(m[w], l[w], v[w]);
#pragma unroll 4
    for (int w = AHEAD; w < s.parts; w++)
        join(ml[2 * w], ml[2 * w + 1], *reinterpret_cast<const f32x4v*>(po + (int64_t)w * a.D));
    const float inv = row_inverse(sum);
#pragma unroll
    for (int c = 0; c < 4; c++) f[c] *= inv;
    store4((TO*)a.out + tok * a.ldo + (int64_t)hq * a.D + d, f);
    if (a.lse && d == 0) a.lse[row] = row_lse(top, sum);
}

// How many parts the longest list of tiles is split into: as many as fill the
// device once (`slots` workgroups), of at least min_tiles each.  (Four tiles of the
// many-row kernel: over 36 sizes 4% above the best of each on average, two 8%, eight
// 6%, sixteen 10%; four a wave of the other: 4%, two 3%, eight 10%.)  More parts
// than that only cost the join (a window of 4096 over six sequences: five parts 25
// us, sixteen 43; nine sequences of chunks: one part 51 us, two 96).  Long lists of
// 64 dimensions, where a CU holds four workgroups, go on to `long_slots` in parts of
// four times as many tiles: over 14 sizes of 300 to 4096 queries 0.73 to 1.03 of the
// time (4 x 300 queries over 8192 keys, 16 heads, 102 us to 74), where 128
// dimensions took 0.78 to 1.40.  All sequences are taken to be as long as max_kv: one
// of 131072 keys among 32 of 500 (32 heads on 8 of 128) stays whole, 1350 us.  More
// parts on the chance of that, sixteen, take it in 133 us, but 64 of 500 with a max_kv
// of 131072 in 103 where this takes 30: workgroups without work hold a CU's LDS while
// they find out.
static void split(AttnDev& d, int64_t max_kv, int rows, int kt, int min_tiles, int slots, int long_slots,
                  int64_t ws_bytes, void* ws) {
    d.row_tiles = (int)(((int64_t)d.max_q * d.G + rows - 1) / rows);
    int64_t seen = max_kv;
    if (d.window > 0)
        seen = std::min(seen, (int64_t)d.window + rows / d.G + d.sinks + 2 * kt);
    const int64_t tiles = std::max<int64_t>(1, (seen + kt - 1) / kt);
    const int64_t blocks = (int64_t)d.row_tiles * d.heads * d.B;
    const int64_t per = (int64_t)d.T * d.q_heads * (d.D + 2) * 4;
    int64_t splits = std::max(std::min(slots / blocks, (tiles + min_tiles - 1) / min_tiles),
                              std::min(long_slots / blocks, tiles / (4 * min_tiles)));
    splits = std::max<int64_t>(1, std::min(splits, std::min<int64_t>(ws_bytes, QGEMV_WS_BYTES) / per));
    d.splits = (int)splits;
    d.split_tiles = (int)((tiles + splits - 1) / splits);
    d.part_o = (float*)ws;
    d.part_ml = d.part_o + (splits > 1 ? (int64_t)d.T * d.q_heads * splits * d.D : 0);
}
template <typename TO, int KT, int ROWS, int LANES>
static void join(const AttnDev& d, hipStream_t st) {
    if (d.splits > 1)
        launch_kernel(k_attn_join<TO, KT, ROWS, LANES>,
                      dim3((unsigned)(((int64_t)d.max_q * d.q_heads * LANES + 255) / 256), (unsigned)d.B),
                      dim3(256), 0, st, d);
}

}  // namespace qgemv
