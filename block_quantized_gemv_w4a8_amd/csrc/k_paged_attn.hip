// k_paged_attn.hip -- attention over a paged cache with causal order, an
// optional sliding window and the first keys that stay visible.
//
// One pass over the keys with the running maximum m and sum l of a softmax
// (Milakov and Gimelshein, "Online normalizer calculation for softmax", 2018):
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
// Two kernels share that.  With many rows (prompts), the waves of a workgroup
// hold 32 rows each and share every K and V tile.  With at most 32 rows (single
// tokens), each wave takes a run of the tiles by itself, with a ring of its own
// for them, and the waves' parts are joined in LDS.  Tiles go from memory
// straight to LDS.  Where there are too few workgroups for the device, the keys
// are split further and a second launch joins the parts.
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
    bool runs;      // 16 keys from a multiple of 16 share a page, and their offsets in it are small
};

// Where keys that are not there and dimensions past the head's come from.
__device__ const uint4 g_zeros[2 * QGEMV_HEAD_DIM_MAX / 16] = {};

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
// scaled: almost every tile after the first few then leaves them alone.
constexpr float kSlack = 8.f;
// The maximum's own weight is 2^kLift.  fp16 ends at 2^16 and holds nothing below
// 2^-24, and o takes the rounded weights where l takes the fp32 ones: with 1 for the
// maximum, a tail of 131071 keys at 2^-25 of it was lost from o alone, 0.36% of the
// row.  With 2^7 the slack ends at 2^15, and what is lost is below 2^-32 of the
// maximum.  bf16 has fp32's range.
template <typename T> constexpr float kLift = std::is_same<T, f16>::value ? 7.f : 0.f;

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

// What a wave holds of its 32 rows, and the steps of a tile of KT keys.
template <typename T, int DP, int KT>
struct Rows {
    typedef Frag<T> F;
    typedef typename F::V V8;
    typedef Lds<DP> L;
    static constexpr int ND = DP / 32, NX = KT / 32, NS = DP / 16;
    static constexpr int CPR = L::CPR, RPI = 64 / CPR;  // chunks of a row; rows of a 1 KB wave load
    V8 qf[NS];
    f32x16 o[ND];
    float m, l;
    float c2;                    // what scores are multiplied by: |scale| log2(e)
    int p, z, p_lo, p_hi, z_hi;  // place and window start of this lane's row, and of the wave's rows
                                 // (p_lo: below every key for a scale of 0, so that hide has every tile)

    // The rows first_row .. first_row + 31 of the block; this lane's is `row`.
    __device__ __forceinline__ void start(const AttnDev& a, const Span& s, int h, int row, int first_row) {
        const int lane = threadIdx.x & 63, half = lane >> 5;
        const int qi = row / a.G, hq = h * a.G + row - qi * a.G;
        p = s.place(qi);
        z = window_start(a, p);
        p_lo = a.scale == 0.f ? INT32_MIN : s.place(min(first_row / a.G, s.i1));
        p_hi = s.place(min((first_row + 31) / a.G, s.i1));
        z_hi = window_start(a, p_hi);
        // (the sign of the scale is moved into q; a scale of 0 is taken in hide, because
        // the -inf of a hidden key times 0 would be NaN)
        c2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
        const T* q = (const T*)a.q + (int64_t)(s.s0 + qi) * a.ldq + (int64_t)hq * a.D;
#pragma unroll
        for (int k = 0; k < NS; k++) {
            const int d = 16 * k + 8 * half;
            V8 f = {};
            if (d < a.D) f = *reinterpret_cast<const V8*>(q + d);
            if (a.scale < 0.f) f = -f;
            qf[k] = f;
        }
#pragma unroll
        for (int d = 0; d < ND; d++) o[d] = f32x16{};
        m = -INFINITY;
        l = 0.f;
    }
    // X^T = K Q^T of the tile at lds + AT.  (Places are constants and the lane's
    // part is formed once: an addition for each read would be a quarter of the
    // vector instructions.)
    template <int AT>
    __device__ __forceinline__ void scores(const char* lds, f32x16 (&x)[NX]) {
        const int half = (threadIdx.x & 63) >> 5, row = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < NX; n++) {
            x[n] = f32x16{};
#pragma unroll
            for (int k = 0; k < NS; k++) {
                const char* at = lds + row * DP * 2 + ((2 * k + half) ^ L::fk(row)) * 16;
                x[n] = F::mfma(*reinterpret_cast<const V8*>(at + AT + 32 * n * DP * 2), qf[k], x[n]);
            }
        }
    }
    // Hides what a row does not see of the tile from key j0 on, of which `there`
    // names the keys that have a page.
    __device__ __forceinline__ void hide(const AttnDev& a, int j0, unsigned long long there, f32x16 (&x)[NX]) {
        const unsigned long long full = KT == 64 ? ~0ull : (1ull << (KT & 63)) - 1;
        if ((there & full) == full && j0 + KT - 1 <= p_lo && (j0 >= z_hi || j0 + KT - 1 < a.sinks)) return;
        if (a.scale == 0.f) {
#pragma unroll
            for (int n = 0; n < NX; n++) x[n] *= 0.f;
        }
        const auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
        // the keys that this lane's row sees, from the first that the lane has on
        const int half = (threadIdx.x & 63) >> 5;
        const unsigned long long seen =
            (there & below(p - j0 + 1) & (~below(z - j0) | below(a.sinks - j0))) >> (4 * half);
        const uint32_t word[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
        for (int n = 0; n < NX; n++)
#pragma unroll
            for (int e = 0; e < 16; e++)
                x[n][e] = word[n] & (1u << (8 * (e / 4) + e % 4)) ? x[n][e] : -INFINITY;
    }
    // Weights from scores, with the running maximum and sum.
    __device__ __forceinline__ void weights(const f32x16 (&x)[NX], V8 (&pf)[2 * NX]) {
        float mt = x[0][0];
#pragma unroll
        for (int n = 0; n < NX; n++)
#pragma unroll
            for (int e = 0; e < 16; e++) mt = fmaxf(mt, x[n][e]);
        mt = max_halves(mt) * c2;
        if (__any(mt > m + kSlack)) {
            const float mn = fmaxf(m, mt);
            const float fix = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            l *= fix;
#pragma unroll
            for (int d = 0; d < ND; d++) o[d] *= fix;
            m = mn;
        }
        const float mu = m == -INFINITY ? 0.f : m - kLift<T>;
        // (l takes a tile's weights at once: one by one those below half of its last
        // bit would be lost, which a tail of 131071 keys at 2^-25 of the maximum is)
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NX; n++)
#pragma unroll
            for (int e = 0; e < 16; e++) {
                const float w = __builtin_amdgcn_exp2f(fmaf(x[n][e], c2, -mu));
                sum += w;
                pf[2 * n + e / 8][e % 8] = (T)w;
            }
        l += sum;
    }
    // After the last tile: l with both halves' keys, and m as what a weight of 1 stands
    // for, by which parts are joined and lse is formed.
    __device__ __forceinline__ void finish() {
        l += __shfl_xor(l, 32);
        m -= kLift<T>;
    }
    // This lane's part of a transposing read: dimensions 32 d .. 32 d + 31, keys 8 w
    // + 4 half .. + 3 of sixteen.
    __device__ __forceinline__ static uint32_t v_part(const char* lds, int d, int w) {
        const int lane = threadIdx.x & 63, half = lane >> 5, g = lane >> 4, i = lane & 15;
        const int key = 8 * w + 4 * half + (i >> 2);
        const int chunk = 4 * d + 2 * (g & 1) + ((i & 3) >> 1);
        return (uint32_t)(uintptr_t)(lmem*)(lds + key * DP * 2 + (chunk ^ L::fv(key)) * 16 + (i & 1) * 8);
    }
    // O^T += V^T P^T of the tile at lds + AT, 16 keys a step: slots 0..3 of a lane
    // are keys 4 half + 0..3 of the step, slots 4..7 the same 8 further on.  Other
    // tiles are on their way to LDS meanwhile, and the compiler would wait for all
    // of them before the reads' builtin; so two steps of 64 dimensions are read,
    // and waited for, at once.
    template <int AT>
    __device__ __forceinline__ void add(const char* lds, const V8 (&pf)[2 * NX]) {
        static_assert(AT + KT * DP * 2 <= 65536, "offsets of a read");
        two_steps<AT, 0>(lds, pf);
        if constexpr (NX == 2) two_steps<AT, 2>(lds, pf);
    }
    template <int AT, int U>
    __device__ __forceinline__ void two_steps(const char* lds, const V8 (&pf)[2 * NX]) {
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
            s16x4 v[2][2][2];   // [step][dimensions][eight keys]
            asm volatile(
                "ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %9 offset:%12\n\t"
                "ds_read_b64_tr_b16 %2, %10 offset:%12\n\tds_read_b64_tr_b16 %3, %11 offset:%12\n\t"
                "ds_read_b64_tr_b16 %4, %8 offset:%13\n\tds_read_b64_tr_b16 %5, %9 offset:%13\n\t"
                "ds_read_b64_tr_b16 %6, %10 offset:%13\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(v[0][0][0]), "=&v"(v[0][0][1]), "=&v"(v[0][1][0]), "=&v"(v[0][1][1]),
                  "=&v"(v[1][0][0]), "=&v"(v[1][0][1]), "=&v"(v[1][1][0]), "=&v"(v[1][1][1])
                : "v"(v_part(lds, d, 0)), "v"(v_part(lds, d, 1)), "v"(v_part(lds, d + 1, 0)),
                  "v"(v_part(lds, d + 1, 1)), "n"(AT + U * 16 * DP * 2), "n"(AT + (U + 1) * 16 * DP * 2)
                : "memory");
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int c = 0; c < 2; c++) o[d + c] = F::mfma(__builtin_bit_cast(V8, v[u][c]), pf[U + u], o[d + c]);
        }
    }
};

// The pages of a tile's keys, from 64 columns of the table at a time (one a
// lane): a tile's columns are within 64 even with a page for every key.  A tile
// whose keys are all there, in pages of whole runs of 16 (a.runs), is addressed
// by scalars: one page and one base a run.  Any other has an offset for every
// key.
template <int DP, int KT>
struct Pages {
    int first = -64, page = -1;            // the lane's column is first + lane
    unsigned long long valid = 0;          // columns with a page of the pool
    int j0;                                // the tile: its first key
    bool runs;                             // whether scalars do
    int64_t off;                           // byte offset of key `lane`, -1 where it is not there

    // The table's first columns, asked for before anything else is known (lengths
    // are on their way meanwhile), and their arrival.  (Chunks gain 1.5 us of 49 by
    // it; single tokens gain nothing.)
    __device__ __forceinline__ void ask(const AttnDev& a, const int32_t* table) {
        const int lane = threadIdx.x & 63;
        first = 0;
        if (lane < a.ldt) page = table[lane];
    }
    __device__ __forceinline__ void arrive(const AttnDev& a) { valid = __ballot(page >= 0 && page < a.n_pages); }

    // Takes up the tile at key j; returns which of its keys are there.
    __device__ __forceinline__ unsigned long long tile(const AttnDev& a, const Span& s, const int32_t* table,
                                                       int j) {
        const int lane = threadIdx.x & 63;
        j0 = j;
        off = -1;
        const int c0 = a.page_shift >= 0 ? j0 >> a.page_shift : j0 / a.page_size;
        const int c1 = a.page_shift >= 0 ? (j0 + KT - 1) >> a.page_shift : (j0 + KT - 1) / a.page_size;
        if (c0 < first || c1 >= first + 64) {
            first = c0;
            page = first + lane < a.ldt ? table[first + lane] : -1;
            arrive(a);   // (the wait for the page is here, not at every tile)
        }
        const unsigned long long need = (2ull << (c1 - c0)) - 1;
        runs = a.runs && j0 + KT <= s.limit && (valid >> (c0 - first) & need) == need;
        if (runs) return ~0ull;
        const int key = j0 + (KT == 64 ? lane : lane & (KT - 1));
        const int c = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
        const int mine = __shfl(page, c - first);
        if (key < s.limit && mine >= 0 && mine < a.n_pages) off = 2 * key_offset(a, mine, key);
        return __ballot(off >= 0);
    }

    // One wave's loads of COUNT KB of the tile's K or V, from row row0 on;
    // `swizzle` says where a row's chunks go.
    template <int COUNT, typename F>
    __device__ __forceinline__ void load(const AttnDev& a, const char* from, int row0, char* to, F swizzle) const {
        constexpr int CPR = Lds<DP>::CPR, RPI = 64 / CPR;
        if (__builtin_expect(runs, 1)) {
            const int lane = threadIdx.x & 63, lr = lane / CPR, lc = lane % CPR;
            constexpr int RUN = COUNT * RPI < 16 ? COUNT : 16 / RPI;   // loads of (part of) a run
            static_assert(COUNT % RUN == 0, "whole runs");
            const uint32_t stride = 2 * (uint32_t)a.token_stride;
#pragma unroll
            for (int r = 0; r < COUNT / RUN; r++) {
                const int key = j0 + row0 + RUN * RPI * r;
                const int pg = __builtin_amdgcn_readlane(page, (key >> a.page_shift) - first);
                const char* base = from + 2 * (pg * a.page_stride + (key & (a.page_size - 1)) * a.token_stride);
#pragma unroll
                for (int c = 0; c < RUN; c++) {
                    const int row = row0 + RUN * RPI * r + RPI * c;
                    uint32_t at = (RPI * c + lr) * stride + 16 * (lc ^ swizzle(row | lr));
                    asm volatile("" : "+v"(at));   // (32 bits to keep, not an address)
                    __builtin_amdgcn_global_load_lds((gmem*)(base + at), (lmem*)(to + row * DP * 2), 16, 0, 0);
                }
            }
            return;
        }
        // (hidden from the compiler, which would form addresses for this branch
        // ahead of the loop over tiles, in registers that the others need)
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int lr = lane / CPR, lc = lane % CPR;
#pragma unroll
        for (int c = 0; c < COUNT; c++) {
            const int row = row0 + RPI * c + lr;
            const int64_t at = __shfl((long long)off, row);
            const int chunk = lc ^ swizzle(row);
            const char* g = from + (at + 16 * chunk);
            g = at >= 0 && 8 * chunk < a.D ? g : (const char*)g_zeros;
            __builtin_amdgcn_global_load_lds((gmem*)g, (lmem*)(to + (row0 + RPI * c) * DP * 2), 16, 0, 0);
        }
    }
};

// Many rows: NW waves of 32 rows each, which share every tile of KT keys, the next
// tile on its way while one is used, and waited for whole.  Bound by a tile's chain
// of loads, scores, weights and products, about 2.2 us at 64 dimensions as at 128
// with two workgroups a CU: the vector and the matrix pipe have about the same work
// (206 and 32 instructions a wave and tile of 64 keys at 128 dimensions) but hardly
// have it at once, the matrix cores being busy 0.47 of the time.  8192 tokens of 32
// heads on 8, causal, take 560 to 600 us with the machine, 920 to 980 TFLOP/s (with
// the LDS places formed for each read, 302 vector instructions, 629 where this took
// 567; with the scores of 32 keys formed beside the weights of the 32 before, 660);
// nine sequences of chunks with a window of 1024 43 us.
template <typename T, typename TO, int DP, int KT, int NW, int OCC>
__global__ __launch_bounds__(64 * NW, OCC) void k_attn_many(const AttnDev a) {
    typedef Rows<T, DP, KT> R;
    typedef Lds<DP> L;
    constexpr int ROWS = 32 * NW;
    constexpr int TILE = KT * DP * 2, BUF = 2 * TILE;  // bytes of a K (or V) tile, and of both
    constexpr int LOADS = KT / R::RPI / NW;            // wave loads of K (and of V) per wave
    static_assert(LOADS >= 1 && KT <= 64, "tile shape");
    extern __shared__ __attribute__((aligned(1024))) char lds[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    // heads first, so that the workgroups of one head meet in one L2; the row
    // tiles with the most keys first
    const int h = blockIdx.x % a.heads;
    const int rest = blockIdx.x / a.heads;
    const int part = rest % a.splits, row_tile = a.row_tiles - 1 - rest / a.splits;
    const int b = blockIdx.y;
    const int32_t* table = a.table + b * a.ldt;
    Pages<DP, KT> pages;
    pages.ask(a, table);
    Span s;
    if (!make_span<KT, ROWS>(a, b, row_tile, part, s)) return;

    // this lane's row, the last one of the block where it has none of its own
    const int first_row = row_tile * ROWS + 32 * wave, r = first_row + (lane & 31);
    const int r_end = (s.i1 + 1) * a.G;
    const int rc = min(r, r_end - 1);
    const bool active = first_row < r_end;
    R w;
    w.start(a, s, h, rc, first_row);
    pages.arrive(a);

    const char* kbase = (const char*)((const T*)a.k + h * a.head_stride);
    const char* vbase = (const char*)((const T*)a.v + h * a.head_stride);
    auto load_tile = [&](int t, char* buf) -> unsigned long long {
        const unsigned long long there = pages.tile(a, s, table, tile_of(s, t) * KT);
        pages.template load<LOADS>(a, kbase, R::RPI * LOADS * wave, buf, L::fk);
        pages.template load<LOADS>(a, vbase, R::RPI * LOADS * wave, buf + TILE, L::fv);
        return there;
    };

    unsigned long long there = 0, there_next = 0;
    if (s.t0 < s.t1) there = load_tile(s.t0, lds);
    QGEMV_WAIT("vmcnt(0)");
    QGEMV_BARRIER();
    auto step = [&](int t, auto at) {
        constexpr int AT = at;
        if (t + 1 < s.t1) there_next = load_tile(t + 1, lds + (BUF - AT));
        const int j0 = tile_of(s, t) * KT;
        if (active && j0 <= w.p_hi && (j0 + KT > window_start(a, w.p_lo) || j0 < a.sinks)) {
            f32x16 x[R::NX];
            typename R::V8 pf[2 * R::NX];
            w.template scores<AT>(lds, x);
            w.hide(a, j0, there, x);
            w.weights(x, pf);
            w.template add<AT + TILE>(lds, pf);
        }
        QGEMV_WAIT("vmcnt(0) lgkmcnt(0)");
        QGEMV_BARRIER();
        there = there_next;
    };
    for (int t = s.t0; t < s.t1; t += 2) {
        step(t, std::integral_constant<int, 0>{});
        if (t + 1 < s.t1) step(t + 1, std::integral_constant<int, BUF>{});
    }
    if (!active) return;
    w.finish();

    bool bad = false;
#pragma unroll
    for (int d = 0; d < R::ND; d++)
#pragma unroll
        for (int e = 0; e < 16; e++) bad |= !(fabsf(w.o[d][e]) < INFINITY);
    bad |= __shfl_xor((int)bad, 32);
    const bool own = r < r_end;
    const int qi = rc / a.G, hq = h * a.G + rc - qi * a.G;
    const int64_t tok = s.s0 + qi, row = tok * a.q_heads + hq;
    if (own && !bad) {
        const int64_t at = row * a.splits + part;
        const float inv = s.parts > 1 ? 1.f : row_scale(w.l);
        TO* out = (TO*)a.out + tok * a.ldo + (int64_t)hq * a.D;
#pragma unroll
        for (int d = 0; d < R::ND; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int d0 = 32 * d + 8 * e + 4 * half;
                if (d0 >= a.D) continue;
                const float f[4] = {w.o[d][4 * e] * inv, w.o[d][4 * e + 1] * inv,
                                    w.o[d][4 * e + 2] * inv, w.o[d][4 * e + 3] * inv};
                if (s.parts > 1) store4(a.part_o + at * a.D + d0, f);
                else store4(out + d0, f);
            }
        if (half == 0) {
            if (s.parts > 1) {
                a.part_ml[2 * at] = w.m;
                a.part_ml[2 * at + 1] = w.l;
            } else if (a.lse) {
                a.lse[row] = row_lse(w.m, w.l);
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
}

// At most 32 rows: each of NW waves takes a run of the tiles.  Its ring holds two
// K and two V tiles; a tile's K makes room for the K after next as soon as the
// scores are formed, and V likewise, so that three of the four are always on
// their way.  Bound by the cache's bytes: 64 sequences of up to 8192 keys take 313
// us, 5.5 TB/s (361 with whole tiles in turn, two to a wave; 256 dimensions, two
// waves a CU, 4.8 TB/s); one short sequence is bound by the chain of lengths, pages,
// keys, 9.6 us.
template <typename T, typename TO, int DP, int NW>
__global__ __launch_bounds__(64 * NW, (NW + 3) / 4) void k_attn_few(const AttnDev a) {
    constexpr int KT = 32, ROWS = 32;
    typedef Rows<T, DP, KT> R;
    typedef Lds<DP> L;
    constexpr int TILE = KT * DP * 2, RING = 4 * TILE;  // bytes of a K (or V) tile, and of a wave's ring
    constexpr int LOADS = KT / R::RPI;                  // wave loads of a tile
    extern __shared__ __attribute__((aligned(1024))) char lds[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, row32 = lane & 31;
    const int h = blockIdx.x % a.heads, part = blockIdx.x / a.heads, b = blockIdx.y;
    const int32_t* table = a.table + b * a.ldt;
    Pages<DP, KT> pages;
    Span s;
    if (!make_span<KT, ROWS>(a, b, 0, part, s)) return;
    const int rows = (s.i1 + 1) * a.G;
    R w;
    w.start(a, s, h, min(row32, rows - 1), 0);

    const char* kbase = (const char*)((const T*)a.k + h * a.head_stride);
    const char* vbase = (const char*)((const T*)a.v + h * a.head_stride);
    char* mine = lds + wave * RING;                     // K, K, V, V
    const int each = (s.t1 - s.t0 + NW - 1) / NW;
    const int t0 = min(s.t0 + wave * each, s.t1), t1 = min(t0 + each, s.t1);
    auto take = [&](int t) { return pages.tile(a, s, table, tile_of(s, t) * KT); };
    auto load_k = [&](int slot) { pages.template load<LOADS>(a, kbase, 0, mine + slot * TILE, L::fk); };
    auto load_v = [&](int slot) { pages.template load<LOADS>(a, vbase, 0, mine + (2 + slot) * TILE, L::fv); };
    if (t0 < t1) {
        unsigned long long there[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (t0 + i >= t1) break;
            there[i] = take(t0 + i);
            load_k(i);
            load_v(i);
        }
        auto step = [&](int t, auto at) {
            constexpr int SLOT = at;
            f32x16 x[R::NX];
            typename R::V8 pf[2 * R::NX];
            // (loads land in their order: K V of this tile, K V of the next, K of the one after)
            const int left = t1 - 1 - t;
            if (left > 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * LOADS) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
            w.template scores<SLOT * TILE>(mine, x);
            QGEMV_WAIT("lgkmcnt(0)");
            const unsigned long long here = there[0];
            there[0] = there[1];
            if (left > 1) {
                there[1] = take(t + 2);
                load_k(SLOT);
            }
            w.hide(a, tile_of(s, t) * KT, here, x);
            w.weights(x, pf);
            if (left > 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * LOADS) : "memory");
            else if (left > 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LOADS) : "memory");
            else QGEMV_WAIT("vmcnt(0)");
            w.template add<(2 + SLOT) * TILE>(mine, pf);
            QGEMV_WAIT("lgkmcnt(0)");
            if (left > 1) load_v(SLOT);
        };
        for (int t = t0; t < t1; t += 2) {
            step(t, std::integral_constant<int, 0>{});
            if (t + 1 < t1) step(t + 1, std::integral_constant<int, 1>{});
        }
        w.finish();
    }

    // the waves' parts of the rows meet in LDS
    constexpr int LD = DP + 4;
    static_assert(32 * LD * 4 <= RING, "a wave's result fits its ring");
    float* po = reinterpret_cast<float*>(mine);
    float* ml = reinterpret_cast<float*>(lds + NW * RING);   // [NW][2][32]
#pragma unroll
    for (int d = 0; d < R::ND; d++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const f32x4v f = {w.o[d][4 * e], w.o[d][4 * e + 1], w.o[d][4 * e + 2], w.o[d][4 * e + 3]};
            *reinterpret_cast<f32x4v*>(po + row32 * LD + 32 * d + 8 * e + 4 * half) = f;
        }
    if (half == 0) {
        ml[wave * 64 + row32] = w.m;
        ml[wave * 64 + 32 + row32] = w.l;
    }
    __syncthreads();
    for (int rr = wave; rr < rows; rr += NW) {
        float top = -INFINITY, sum = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NW; i++) top = fmaxf(top, ml[i * 64 + rr]);
#pragma unroll
        for (int i = 0; i < NW; i++) {
            const float mi = ml[i * 64 + rr];
            const float fix = mi == top ? 1.f : exp2f(mi - top);
            sum += ml[i * 64 + 32 + rr] * fix;
            const float* src = reinterpret_cast<const float*>(lds + i * RING) + rr * LD;
#pragma unroll
            for (int c = 0; c < DP / 64; c++) f[c] += src[lane + 64 * c] * fix;
        }
        bool bad = false;
#pragma unroll
        for (int c = 0; c < DP / 64; c++) bad |= !(fabsf(f[c]) < INFINITY);
        const int i = rr / a.G, hh = h * a.G + rr - i * a.G;
        if (__any(bad))
            attn_row<T, KT>(a, s, table, i, hh, a.scale * 1.4426950408889634f, f, top, sum);
        put_row<TO>(a, s, part, i, hh, f, top, sum);
    }
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
    const float inv = row_scale(sum);
#pragma unroll
    for (int c = 0; c < 4; c++) f[c] *= inv;
    store4((TO*)a.out + tok * a.ldo + (int64_t)hq * a.D + d, f);
    if (a.lse && d == 0) a.lse[row] = row_lse(top, sum);
}

// How many parts the longest list of tiles is split into: as many as fill the
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

template <typename T, typename TO, int DP, int KT, int OCC>
static void launch_many(AttnDev d, const AttnArgs& a, hipStream_t st) {
    constexpr int NW = 4, ROWS = 32 * NW;
    split(d, a.max_kv, ROWS, KT, 4, 256 * OCC, DP == 64 ? 1024 : 0, a.ws_bytes, a.ws);
    launch_kernel(k_attn_many<T, TO, DP, KT, NW, OCC>,
                  dim3((unsigned)(d.heads * d.splits * d.row_tiles), (unsigned)d.B), dim3(64 * NW),
                  2 * 2 * KT * DP * 2, st, d);
    join<TO, KT, ROWS, DP / 4>(d, st);
}
template <typename T, typename TO, int DP, int NW>
static void launch_few(AttnDev d, const AttnArgs& a, hipStream_t st) {
    split(d, a.max_kv, 32, 32, 4 * NW, 256, 0, a.ws_bytes, a.ws);
    launch_kernel(k_attn_few<T, TO, DP, NW>, dim3((unsigned)(d.heads * d.splits), (unsigned)d.B),
                  dim3(64 * NW), NW * (4 * 32 * DP * 2 + 256), st, d);
    join<TO, 32, 32, DP / 4>(d, st);
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
            d.runs = (d.D == 64 || d.D == 128 || d.D == 256) && d.page_shift >= 4 && d.token_stride < (1 << 26);
            if (few) {
                if (d.D <= 64) launch_few<T, TO, 64, 8>(d, a, st);
                else if (d.D <= 128) launch_few<T, TO, 128, 4>(d, a, st);
                else launch_few<T, TO, 256, 2>(d, a, st);
            } else {
                if (d.D <= 64) launch_many<T, TO, 64, 64, 2>(d, a, st);
                else if (d.D <= 128) launch_many<T, TO, 128, 64, 2>(d, a, st);
                else launch_many<T, TO, 256, 32, 1>(d, a, st);
            }
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
