// k_paged_attn.hip -- attention over a paged cache with causal order, an
// optional sliding window and the first keys that stay visible.
//
// One pass over the keys with the running maximum m and sum l of a softmax:
// for each tile of keys, where max x exceeds m, o and l are scaled by
// exp(m - m') and m becomes m'; then exp(x - m) v and exp(x - m) are added.
//
// The rows of a (sequence, cache head) are its queries times the G query heads
// that share the cache head, row r = query r / G, head r % G, so that one read
// of a key serves all of them.  A wave holds 32 rows.  It forms X^T = K Q^T
// with 32x32x16 matrix instructions (keys down, rows across), so a lane owns
// half of the keys of one row: maximum and sum are per lane with one exchange
// between the two halves of the wave, and the weights, rounded to the cache's
// type, already are the B operand of O^T += V^T P^T when the keys of a 16-deep
// step are taken in the order in which X^T left them.  V^T comes from the
// row-major V tile through the transposing LDS read.
//
// Two kernels from one template.  With many rows (prompts), the waves of a
// workgroup hold 32 rows each and share every K and V tile.  With at most 32
// rows (single tokens), each wave takes tiles of its own and the waves' parts
// are joined in LDS.  Tiles go from memory straight to LDS, the next one while
// this one is used.  Where there are too few workgroups for the device, the
// keys are split further and a second launch joins the parts.
#include <algorithm>

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

template <typename T> struct Frag;
template <> struct Frag<bf16> {
    typedef bf16x8 V;
    static __device__ __forceinline__ f32x16 mfma(V a, V b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Frag<f16> {
    typedef f16x8 V;
    static __device__ __forceinline__ f32x16 mfma(V a, V b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

struct AttnDev {
    const void *q, *k, *v;
    void* out;
    float *lse, *part_o, *part_ml;
    const int32_t *q_start, *kv_len, *table;
    int64_t ldq, ldo, ldt, page_stride, token_stride, head_stride;
    int T, q_heads, heads, G, D, B, max_q, n_pages, page_size, page_shift, window, sinks;
    int row_tiles, splits, split_tiles;
    float scale;
};

// Where keys that are not there and dimensions past the head's come from.
__device__ const uint4 g_zeros[2 * QGEMV_HEAD_DIM_MAX / 16] = {};

// The queries of a sequence and the keys that a block of its rows sees, as a
// list of tiles: those of the sinks, then those from the window's start.
struct Span {
    int s0, n, kv;          // first query, queries, keys
    int i0, i1;             // queries of the block
    int limit;              // keys that the table can hold
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
    s.limit = (int)min(a.ldt * a.page_size, (int64_t)0x7fffff00);
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

// One row over one part of its keys, by one wave: a key to a lane for the
// scores, then the dimensions over the lanes.  It touches no key that the row
// does not see, and stands in for the matrix path where a value of an unseen
// key that is not finite (0 * inf) has spoilt the row's sum.
template <typename T, int KT>
__device__ void attn_row(const AttnDev& a, const Span& s, const int32_t* table, int i, int hq,
                         float c2, float (&o)[4], float& m, float& l) {
    const int lane = threadIdx.x & 63;
    const int h = hq / a.G, p = s.place(i), z = window_start(a, p);
    const T* q = (const T*)a.q + (int64_t)(s.s0 + i) * a.ldq + (int64_t)hq * a.D;
    const T* k = (const T*)a.k + h * a.head_stride;
    const T* v = (const T*)a.v + h * a.head_stride;
    m = -INFINITY;
    l = 0.f;
    for (int c = 0; c < 4; c++) o[c] = 0.f;
    for (int t = s.t0; t < s.t1; t++) {
        const int j = tile_of(s, t) * KT + lane;
        int64_t at = -1;
        if (lane < KT && j <= p && (j >= z || j < a.sinks)) {
            const int page = page_of(a, table, j, s.limit);
            if (page >= 0 && page < a.n_pages) at = key_offset(a, page, j);
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
            x *= c2;
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
        for (int c = 0; c < 4; c++) o[c] *= fix;
        for (int u = 0; u < KT; u++) {
            const int64_t tat = __shfl((long long)at, u);
            const float tp = __shfl(pr, u);
            if (tat < 0) continue;
            for (int c = 0; c < 4; c++)
                if (lane + 64 * c < a.D) o[c] = fmaf(tp, (float)v[tat + lane + 64 * c], o[c]);
        }
    }
}

// Four consecutive values of a row of the result, or of a part of it.
template <typename TO>
__device__ __forceinline__ void put4(TO* p, const float (&f)[4]) {
    alignas(16) TO e[4];
#pragma unroll
    for (int i = 0; i < 4; i++) e[i] = (TO)f[i];
    if constexpr (sizeof(TO) == 4) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(e);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(e);
}
// m is in units of log2; 1 / l of a row that saw nothing is 0.
__device__ __forceinline__ float row_scale(float l) { return l != 0.f ? 1.f / l : 0.f; }
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
    const float inv = row_scale(l);
    TO* out = (TO*)a.out + t * a.ldo + (int64_t)hq * a.D;
    for (int c = 0; c < 4; c++)
        if (lane + 64 * c < a.D) out[lane + 64 * c] = (TO)(o[c] * inv);
    if (a.lse && lane == 0) a.lse[row] = row_lse(m, l);
}

// The weights may grow to 2^kSlack of the running maximum's before o and l are
// scaled: almost every tile after the first few then leaves them alone.  2^8
// stays far inside fp16, and the weights' relative precision is the same.
constexpr float kSlack = 8.f;

template <int DP> struct Lds {
    static constexpr int CPR = DP / 8;                 // 16-byte chunks of a row
    // Chunk c of row r sits at place c ^ f(r) of the row.  K: the 32 rows of a
    // fragment's column of chunks fall on all places of 256 bytes.  V: the four
    // rows times 64 bytes of a transposing read do.
    static __device__ __forceinline__ int fk(int r) { return DP == 64 ? (r >> 1) & 7 : r & 15; }
    static __device__ __forceinline__ int fv(int r) {
        return DP == 64 ? ((r >> 1) & 1) << 2 : ((r & 3) << 2) | ((r >> 2) & 3);
    }
};

#define QGEMV_WAIT_LOADS() asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory")
#define QGEMV_BARRIER()                    \
    do {                                   \
        __builtin_amdgcn_s_barrier();      \
        asm volatile("" ::: "memory");     \
    } while (0)

// NW waves; BYKEY: each wave takes every NW-th tile for the same 32 rows, else
// each wave has 32 rows of its own and all share every tile of KT keys.
template <typename T, typename TO, int DP, int KT, int NW, bool BYKEY, int OCC>
__global__ __launch_bounds__(64 * NW, OCC) void k_attn(const AttnDev a) {
    typedef Frag<T> F;
    typedef typename F::V V8;
    typedef Lds<DP> L;
    constexpr int ROWS = BYKEY ? 32 : 32 * NW;
    constexpr int CPR = L::CPR, RPI = 64 / CPR;        // rows of a 1 KB wave load
    constexpr int TILE = KT * DP * 2;                  // bytes of a K (or V) tile
    constexpr int BUF = 2 * TILE;
    constexpr int LOADS = KT / RPI / (BYKEY ? 1 : NW); // wave loads of K (and of V) per wave
    constexpr int ND = DP / 32, NX = KT / 32, NS = DP / 16;
    static_assert(LOADS >= 1 && KT <= 64, "tile shape");
    extern __shared__ __attribute__((aligned(1024))) char lds[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, row32 = lane & 31;
    // heads first, so that the workgroups of one head meet in one L2; the row
    // tiles with the most keys first
    const int h = blockIdx.x % a.heads;
    const int rest = blockIdx.x / a.heads;
    const int part = rest % a.splits, row_tile = a.row_tiles - 1 - rest / a.splits;
    const int b = blockIdx.y;
    Span s;
    if (!make_span<KT, ROWS>(a, b, row_tile, part, s)) return;
    const int32_t* table = a.table + b * a.ldt;

    // this lane's row, the last one of the block where it has none of its own
    const int r = row_tile * ROWS + (BYKEY ? 0 : 32 * wave) + row32;
    const int r_end = (s.i1 + 1) * a.G;
    const int rc = min(r, r_end - 1);
    const int qi = rc / a.G, hq = h * a.G + rc - qi * a.G;
    const int p = s.place(qi), z = window_start(a, p);
    const int first_row = row_tile * ROWS + (BYKEY ? 0 : 32 * wave);
    const bool active = first_row < r_end;
    const int p_lo = s.place(min(first_row / a.G, s.i1));
    const int p_hi = s.place(min((first_row + 31) / a.G, s.i1));
    const int z_hi = window_start(a, p_hi);

    // x2 = |scale| log2(e) (q . k), the sign of the scale moved into q
    const float c2 = fabsf(a.scale) * 1.4426950408889634f;
    V8 qf[NS];
    {
        const T* q = (const T*)a.q + (int64_t)(s.s0 + qi) * a.ldq + (int64_t)hq * a.D;
#pragma unroll
        for (int k = 0; k < NS; k++) {
            const int d = 16 * k + 8 * half;
            V8 f = {};
            if (d < a.D) f = *reinterpret_cast<const V8*>(q + d);
            if (a.scale < 0.f) f = -f;
            qf[k] = f;
        }
    }

    char* mine = lds + (BYKEY ? wave * 2 * BUF : 0);
    const int step = BYKEY ? NW : 1;
    int t = s.t0 + (BYKEY ? wave : 0);

    // lane `x` holds the page, then the offset, of key x of the tile to come
    const int key_lane = KT == 64 ? lane : lane & (KT - 1);
    auto pages = [&](int tt) {
        return tt < s.t1 ? page_of(a, table, tile_of(s, tt) * KT + key_lane, s.limit) : -1;
    };
    const char* kbase = (const char*)((const T*)a.k + h * a.head_stride);
    const char* vbase = (const char*)((const T*)a.v + h * a.head_stride);
    const int lr = lane / CPR, lc = lane % CPR;        // row and place of this lane in a wave load
    auto load_tile = [&](int tt, int page, char* buf) -> unsigned long long {
        const bool there = page >= 0 && page < a.n_pages;
        const int64_t off = there ? 2 * key_offset(a, page, tile_of(s, tt) * KT + key_lane) : -1;
#pragma unroll
        for (int c = 0; c < LOADS; c++) {
            const int row0 = RPI * (c + (BYKEY ? 0 : LOADS * wave));
            const int row = row0 + lr;
            const int64_t at = __shfl((long long)off, row);
            const int ck = lc ^ L::fk(row), cv = lc ^ L::fv(row);
            const char* gk = at >= 0 && 8 * ck < a.D ? kbase + at + 16 * ck : (const char*)g_zeros;
            const char* gv = at >= 0 && 8 * cv < a.D ? vbase + at + 16 * cv : (const char*)g_zeros;
            __builtin_amdgcn_global_load_lds((gmem*)gk, (lmem*)(buf + row0 * DP * 2), 16, 0, 0);
            __builtin_amdgcn_global_load_lds((gmem*)gv, (lmem*)(buf + TILE + row0 * DP * 2), 16, 0, 0);
        }
        return __ballot(there);
    };

    f32x16 o[ND] = {};
    float m = -INFINITY, l = 0.f;

    int page_next = pages(t);
    unsigned long long there = 0, there_next = 0;
    int buf = 0;
    if (t < s.t1) there = load_tile(t, page_next, mine);
    page_next = pages(t + step);
    QGEMV_WAIT_LOADS();
    if (!BYKEY) QGEMV_BARRIER();

    for (; t < s.t1; t += step) {
        if (t + step < s.t1) there_next = load_tile(t + step, page_next, mine + (buf ^ BUF));
        page_next = pages(t + 2 * step);
        const char* kt = mine + buf;
        const char* vt = mine + buf + TILE;
        const int j0 = tile_of(s, t) * KT;
        const bool any = active && j0 <= p_hi &&
                         (j0 + KT > window_start(a, p_lo) || j0 < a.sinks);
        if (any) {
            f32x16 x[NX];
#pragma unroll
            for (int n = 0; n < NX; n++) {
                x[n] = f32x16{};
#pragma unroll
                for (int k = 0; k < NS; k++) {
                    const int row = 32 * n + row32;
                    const int place = (2 * k + half) ^ L::fk(row);
                    const V8 kf = *reinterpret_cast<const V8*>(kt + row * DP * 2 + place * 16);
                    x[n] = F::mfma(kf, qf[k], x[n]);
                }
            }
            const unsigned long long full = KT == 64 ? ~0ull : (1ull << (KT & 63)) - 1;
            const bool all = (there & full) == full && j0 + KT - 1 <= p_lo &&
                             (j0 >= z_hi || j0 + KT - 1 < a.sinks);
            if (!all) {
#pragma unroll
                for (int n = 0; n < NX; n++)
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const int key = 32 * n + 8 * (e / 4) + 4 * half + e % 4;
                        const int j = j0 + key;
                        const bool seen = j <= p && (j >= z || j < a.sinks) && (there >> key & 1);
                        x[n][e] = seen ? x[n][e] : -INFINITY;
                    }
            }
            float mt = x[0][0];
#pragma unroll
            for (int n = 0; n < NX; n++)
#pragma unroll
                for (int e = 0; e < 16; e++) mt = fmaxf(mt, x[n][e]);
            mt = fmaxf(mt, __shfl_xor(mt, 32)) * c2;
            if (__any(mt > m + kSlack)) {
                const float mn = fmaxf(m, mt);
                const float fix = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
                l *= fix;
#pragma unroll
                for (int d = 0; d < ND; d++) o[d] *= fix;
                m = mn;
            }
            const float mu = m == -INFINITY ? 0.f : m;
            V8 pf[2 * NX];
#pragma unroll
            for (int n = 0; n < NX; n++)
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const float w = __builtin_amdgcn_exp2f(fmaf(x[n][e], c2, -mu));
                    l += w;
                    pf[2 * n + e / 8][e % 8] = (T)w;
                }
            // O^T += V^T P^T, 16 keys a step: slots 0..3 of a lane are keys
            // 4 half + 0..3 of the step, slots 4..7 the same 8 further on
            const int g = lane >> 4, i = lane & 15;
#pragma unroll
            for (int u = 0; u < 2 * NX; u++)
#pragma unroll
                for (int d = 0; d < ND; d++) {
                    s16x4 part2[2];
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        const int key = 16 * u + 8 * w + 4 * half + (i >> 2);
                        const int chunk = 4 * d + 2 * (g & 1) + ((i & 3) >> 1);
                        const char* at = vt + key * DP * 2 + (chunk ^ L::fv(key)) * 16 + (i & 1) * 8;
                        part2[w] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lmem4*)at);
                    }
                    const V8 vf = __builtin_bit_cast(V8, part2);
                    o[d] = F::mfma(vf, pf[u], o[d]);
                }
        }
        QGEMV_WAIT_LOADS();
        if (!BYKEY) QGEMV_BARRIER();
        buf ^= BUF;
        there = there_next;
    }
    l += __shfl_xor(l, 32);

    if constexpr (!BYKEY) {
        if (!active) return;
        bool bad = false;
#pragma unroll
        for (int d = 0; d < ND; d++)
#pragma unroll
            for (int e = 0; e < 16; e++) bad |= !(fabsf(o[d][e]) < INFINITY);
        bad |= __shfl_xor((int)bad, 32);
        const bool own = r < r_end;
        const int64_t tok = s.s0 + qi, row = tok * a.q_heads + hq;
        if (own && !bad) {
            const int64_t at = row * a.splits + part;
            const float inv = s.parts > 1 ? 1.f : row_scale(l);
            TO* out = (TO*)a.out + tok * a.ldo + (int64_t)hq * a.D;
#pragma unroll
            for (int d = 0; d < ND; d++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int d0 = 32 * d + 8 * e + 4 * half;
                    if (d0 >= a.D) continue;
                    const float f[4] = {o[d][4 * e] * inv, o[d][4 * e + 1] * inv,
                                        o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv};
                    if (s.parts > 1) put4(a.part_o + at * a.D + d0, f);
                    else put4(out + d0, f);
                }
            if (half == 0) {
                if (s.parts > 1) {
                    a.part_ml[2 * at] = m;
                    a.part_ml[2 * at + 1] = l;
                } else if (a.lse) {
                    a.lse[row] = row_lse(m, l);
                }
            }
        }
        for (unsigned todo = (unsigned)__ballot(own && bad); todo; todo &= todo - 1) {
            const int rr = first_row + __builtin_ctz(todo);
            const int i = rr / a.G, hh = h * a.G + rr - i * a.G;
            float ro[4], rm, rl;
            attn_row<T, KT>(a, s, table, i, hh, a.scale * 1.4426950408889634f, ro, rm, rl);
            put_row<TO>(a, s, part, i, hh, ro, rm, rl);
        }
    } else {
        // the waves' parts of the 32 rows meet in LDS
        constexpr int LD = DP + 4;
        float* po = reinterpret_cast<float*>(mine);
        float* ml = reinterpret_cast<float*>(lds + NW * 2 * BUF);   // [NW][2][32]
        static_assert(32 * LD * 4 <= 2 * BUF, "a wave's result fits its tiles");
#pragma unroll
        for (int d = 0; d < ND; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const f32x4v f = {o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
                *reinterpret_cast<f32x4v*>(po + row32 * LD + 32 * d + 8 * e + 4 * half) = f;
            }
        if (half == 0) {
            ml[wave * 64 + row32] = m;
            ml[wave * 64 + 32 + row32] = l;
        }
        __syncthreads();
        const int rows = min(32, r_end - row_tile * ROWS);
        for (int rr = wave; rr < rows; rr += NW) {
            float top = -INFINITY, sum = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < NW; w++) top = fmaxf(top, ml[w * 64 + rr]);
            for (int w = 0; w < NW; w++) {
                const float mw = ml[w * 64 + rr];
                const float fix = mw == top ? 1.f : exp2f(mw - top);
                sum += ml[w * 64 + 32 + rr] * fix;
                const float* src = reinterpret_cast<const float*>(lds + w * 2 * BUF) + rr * LD;
#pragma unroll
                for (int c = 0; c < DP / 64; c++) f[c] += src[lane + 64 * c] * fix;
            }
            bool bad = false;
#pragma unroll
            for (int c = 0; c < DP / 64; c++) bad |= !(fabsf(f[c]) < INFINITY);
            const int rg = row_tile * ROWS + rr;
            const int i = rg / a.G, hh = h * a.G + rg - i * a.G;
            if (__any(bad))
                attn_row<T, KT>(a, s, table, i, hh, a.scale * 1.4426950408889634f, f, top, sum);
            put_row<TO>(a, s, part, i, hh, f, top, sum);
        }
    }
}

// Joins the parts of the rows whose keys were split: one wave a row.
template <typename TO, int KT, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join(const AttnDev a) {
    const int lane = threadIdx.x & 63;
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6);      // query and head of the sequence
    const int b = blockIdx.y;
    const int i = r / a.q_heads, hq = r - i * a.q_heads, h = hq / a.G;
    if (i >= a.max_q) return;
    Span s;
    const int row_tile = (i * a.G + hq - h * a.G) / ROWS;
    if (!make_span<KT, ROWS>(a, b, row_tile, 0, s) || i >= s.n || s.parts == 1) return;
    const int64_t row = (int64_t)(s.s0 + i) * a.q_heads + hq;
    const float* ml = a.part_ml + 2 * row * a.splits;
    const float* po = a.part_o + row * a.splits * a.D;
    float top = -INFINITY, sum = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < s.parts; w++) top = fmaxf(top, ml[2 * w]);
    for (int w = 0; w < s.parts; w++) {
        const float mw = ml[2 * w];
        const float fix = mw == top ? 1.f : exp2f(mw - top);
        sum += ml[2 * w + 1] * fix;
        for (int c = 0; c < 4; c++)
            if (lane + 64 * c < a.D) f[c] += po[(int64_t)w * a.D + lane + 64 * c] * fix;
    }
    s.parts = 1;
    put_row<TO>(a, s, 0, i, hq, f, top, sum);
}

template <typename T, typename TO, int DP, int KT, int NW, bool BYKEY, int OCC>
static void launch_one(AttnDev d, int64_t max_kv, int64_t ws_bytes, void* ws, hipStream_t st) {
    constexpr int ROWS = BYKEY ? 32 : 32 * NW;
    constexpr unsigned smem = 2 * 2 * KT * DP * 2 * (BYKEY ? NW : 1) + (BYKEY ? NW * 256 : 0);
    d.row_tiles = (int)(((int64_t)d.max_q * d.G + ROWS - 1) / ROWS);
    // the longest list of tiles, and how many parts of it fill the device
    int64_t seen = max_kv;
    if (d.window > 0)
        seen = std::min(seen, (int64_t)d.window + ROWS / d.G + std::min(d.sinks, d.window) + 2 * KT);
    const int64_t tiles = std::max<int64_t>(1, (seen + KT - 1) / KT);
    const int64_t blocks = (int64_t)d.row_tiles * d.heads * d.B;
    const int64_t min_tiles = BYKEY ? 4 * NW : 8;
    int64_t splits = std::min((768 + blocks - 1) / blocks, (tiles + min_tiles - 1) / min_tiles);
    const int64_t per = (int64_t)d.T * d.q_heads * (d.D + 2) * 4;
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, ws_bytes / per));
    d.splits = (int)splits;
    d.split_tiles = (int)((tiles + splits - 1) / splits);
    d.part_o = (float*)ws;
    d.part_ml = d.part_o + (splits > 1 ? (int64_t)d.T * d.q_heads * splits * d.D : 0);
    launch_kernel(k_attn<T, TO, DP, KT, NW, BYKEY, OCC>,
                  dim3((unsigned)(d.heads * d.splits * d.row_tiles), (unsigned)d.B), dim3(64 * NW),
                  smem, st, d);
    if (splits > 1)
        launch_kernel(k_attn_join<TO, KT, ROWS>,
                      dim3((unsigned)(((int64_t)d.max_q * d.q_heads + 3) / 4), (unsigned)d.B),
                      dim3(256), 0, st, d);
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
    d.page_shift = (a.c.page_size & (a.c.page_size - 1)) == 0 ? __builtin_ctz(a.c.page_size) : -1;
    const bool few = (int64_t)a.max_q * d.G <= 32;
    with_type16(a.c.type, [&](auto t) {
        with_type(a.out_type, [&](auto to) {
            using T = decltype(t);
            using TO = decltype(to);
#define QGEMV_ATTN(DP, KT, NW, BYKEY, OCC) \
    launch_one<T, TO, DP, KT, NW, BYKEY, OCC>(d, a.max_kv, a.ws_bytes, a.ws, st)
            if (few) {
                if (d.D <= 64) QGEMV_ATTN(64, 32, 4, true, 2);
                else if (d.D <= 128) QGEMV_ATTN(128, 32, 4, true, 1);
                else QGEMV_ATTN(256, 32, 2, true, 1);
            } else {
                if (d.D <= 64) QGEMV_ATTN(64, 64, 4, false, 2);
                else if (d.D <= 128) QGEMV_ATTN(128, 64, 4, false, 2);
                else QGEMV_ATTN(256, 32, 4, false, 1);
            }
#undef QGEMV_ATTN
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
