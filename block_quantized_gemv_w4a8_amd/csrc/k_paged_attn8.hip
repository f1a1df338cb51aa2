// k_paged_attn8.hip -- attention over a paged cache of int8 codes with one scale a
// row, with causal order, an optional sliding window and the first keys that stay
// visible.
//
// With codes ck, cv and scales sk, sv: x_j = scale sk_j (q . ck_j), m their
// largest, w_j = exp(x_j - m), out = sum w_j sv_j cv_j / sum w_j, in one pass over
// the keys with the running maximum and sum of a softmax.  Codes are whole numbers
// that fp16 holds, so they go to the fp16 matrix cores exactly and the scales are
// taken in fp32 on both sides of them: a key's multiplies its score, a value's its
// weight.  The weight is then rounded to fp16, or to two that add up to it, with factors
// of two that keep it in fp16's range (kLift, and the largest scale that the row has seen).
//
// Rows, tiles and their order are those of the attention over 16-bit values: the
// queries of a sequence times the G query heads of a cache head, 32 rows a wave, X^T
// = K Q^T (keys down, rows across), O^T += V^T P^T.
#include <utility>

#include "qgemv_attn.h"

namespace qgemv {

struct Attn8Dev : AttnDev {     // (strides of codes in bytes)
    const float *ks, *vs;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    bool by_die;
    uint32_t page_bytes, slot_bytes, scale_page, scale_slot;   // the strides where `runs` holds
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

// A code and a half are one number: 1024 + (code + 128) in fp16 is 0x6400 with the
// code's byte, its top bit turned over, in the low bits; 1152 less is the code.
// Five instructions for four codes.
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) const f16x8 lmem16;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// (loads that are known to be global: others count as LDS's too, which then are waited for all at once)
typedef __attribute__((address_space(1))) const u32x4 gmem16;
typedef __attribute__((address_space(1))) const float gmemf;
__device__ __forceinline__ f16x8 halves(uint32_t lo, uint32_t hi) {
    const f16x2 off = {(f16)-1152.f, (f16)-1152.f};
    const uint32_t w[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
    union { f16x2 h[4]; f16x8 v; } r;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        r.h[2 * i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04010400u)) + off;
        r.h[2 * i + 1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04030402u)) + off;
    }
    return r.v;
}
__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// What weights may grow to before o and l are scaled, and the weight of the maximum:
// 2^7 to 2^15, so that fp16 (2^-24 to 2^16) holds what is above 2^-32 of a row's
// largest.  A weight times a value's scale is held there by 2^-r, 2^r the first power
// of two that no seen scale of the row exceeds; l takes the same factor, which so
// falls out of o / l.  r is kept as a float's exponent field, in -60 .. 60 (larger
// scales overflow and are left to attn8_row; what smaller ones add may be lost).
constexpr float kSlack8 = 8.f, kLift8 = 7.f;
constexpr int kLeast = 127 - 60, kMost = 127 + 60;

// Kinds of instructions for the order that the scheduler is asked for.
constexpr int kValu = 0x402, kMfma = 0x8, kDsRead = 0x100;

// Where chunks of 16 bytes of a row stand: chunk c of row r of an LDS tile at place c
// ^ f(r) of the row.  Codes (rows of DP bytes): 16 lanes that read one chunk of
// 16 keys, and the 16 keys times 32 bytes of a transposing read by half waves, fall on
// all places of 256 bytes.
template <int DP> struct Place8 {
    static __device__ __forceinline__ int k(int r) { return DP == 64 ? (r >> 2) & 3 : DP == 128 ? (r >> 1) & 7 : r & 15; }
    static __device__ __forceinline__ int v(int r) {
        return DP == 64 ? (r >> 3 & 1) << 1 : DP == 128 ? (r >> 1 & 1) << 1 | (r >> 3 & 1) << 2 : (r & 3) << 1 | (r >> 3 & 1) << 3;
    }
};
// Halves (rows of 2 DP bytes): the same for reads, and for writes of a row's
// chunks by every second.
template <int DP> struct Place16 {
    static __device__ __forceinline__ int k(int r) { return DP == 64 ? (r >> 1) & 7 : r & 15; }
    static __device__ __forceinline__ int v(int r) { return DP == 64 ? (r >> 1 & 1) * 5 : (r & 3) << 2 | ((r >> 2 ^ r) & 3); }
};

// x[e] times what lane e of the lane's row of sixteen holds.
template <int E>
__device__ __forceinline__ float lane_of_row(float s) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), 0x150 + E, 0xf, 0xf, true));
}
template <int E>
__device__ __forceinline__ float times_lane(float x, float s) {
    float y = lane_of_row<E>(s) * x;
    asm("" : "+v"(y));   // (in pairs the products would not take the broadcast in)
    return y;
}
template <int... E>
__device__ __forceinline__ void times_lanes(f32x16& x, float s, std::integer_sequence<int, E...>) {
    ((x[E] = times_lane<E>(x[E], s)), ...);
}
template <int USE>
__device__ __forceinline__ void times_lanes(f32x16& x, float s) {
    asm("; use %1" : "+v"(s) : "n"(USE));   // (the broadcasts are this use's own, not shared with another's in registers)
    times_lanes(x, s, std::make_integer_sequence<int, 16>{});
}

// (fmaxf would first make each of them quiet, one instruction more a value)
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}

// What a wave holds of its 32 rows, and the steps of a tile of KT keys.
template <int DP, int KT>
struct Rows8 {
    static constexpr int ND = DP / 32, NX = KT / 32, NS = DP / 16;
    f16x8 qf[NS];
    f32x16 o[ND];
    float m, l;
    int r;                       // exponent field of the scales' factor
    float r_min;                 // the least factor of the wave's rows
    float mu;                    // what is taken from a score (times c2) before its exponential
    float c2;                    // what scores are multiplied by: |scale| log2(e), and q's factor
    int p, z, p_lo, p_hi, z_lo, z_hi;  // place and window start of this lane's row, and of the wave's rows
                                 // (p_lo: below every key for a scale of 0, so that scaled looks at every tile)

    // The rows first_row .. first_row + 31 of the block; this lane's is `row`.  A
    // lane has, of each 32 dimensions, the 16 from `first` on: in two runs of 8
    // that lie together (JOINED, as a read of 16 codes leaves them) or 16 apart.  ask()
    // sends for q's values, start() takes them: between the two the first tiles are sent for.
    template <typename T> struct Query {
        typedef T V8 __attribute__((ext_vector_type(8)));
        V8 in[NS];
    };
    template <typename T, bool JOINED>
    __device__ __forceinline__ Query<T> ask(const AttnDev& a, const Span& s, int h, int row, int first_row) {
        typedef typename Query<T>::V8 V8;
        const int half = (threadIdx.x & 63) >> 5;
        const int qi = row / a.G, hq = h * a.G + row - qi * a.G;
        p = s.place(qi);
        z = window_start(a, p);
        p_lo = a.scale == 0.f ? INT32_MIN : s.place(min(first_row / a.G, s.i1));
        p_hi = s.place(min((first_row + 31) / a.G, s.i1));
        z_lo = window_start(a, s.place(min(first_row / a.G, s.i1)));
        z_hi = window_start(a, p_hi);
        const T* q = (const T*)a.q + (int64_t)(s.s0 + qi) * a.ldq + (int64_t)hq * a.D;
        Query<T> r;
#pragma unroll
        for (int k = 0; k < NS; k++) {
            const int d = JOINED ? 32 * (k / 2) + 16 * half + 8 * (k % 2) : 16 * k + 8 * half;
            r.in[k] = V8{};
            if (d < a.D) r.in[k] = *reinterpret_cast<const V8*>(q + d);
        }
        return r;
    }
    template <typename T>
    __device__ __forceinline__ void start(const AttnDev& a, const Query<T>& query) {
        const auto& in = query.in;
        // (the sign of the scale is moved into q; a scale of 0 is taken in scaled, because
        // the -inf of a hidden key times 0 would be NaN)
        c2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
        float f = a.scale < 0.f ? -1.f : 1.f;
        if constexpr (std::is_same<T, bf16>::value) {
            // bf16 as fp16 times a power of two that takes the row's largest value to 2^14
            // .. 2^15: eight bits of each value then stand down to 2^-31 of it, and what is
            // below 2^-39 of it is lost
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < NS; k++)
#pragma unroll
                for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf((float)in[k][e]));
            top = fmaxf(top, __shfl_xor(top, 32));
            // (rows of zeros, rows below 2^-99 and what is not finite: a factor within the range)
            int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23);
            e = e == 255 ? 127 + 14 : max(e, 27);
            f *= __builtin_bit_cast(float, (uint32_t)(127 + 14 + 127 - e) << 23);
            c2 *= __builtin_bit_cast(float, (uint32_t)(e - 14) << 23);
        }
#pragma unroll
        for (int k = 0; k < NS; k++)
#pragma unroll
            for (int e = 0; e < 8; e++) qf[k][e] = (f16)((float)in[k][e] * f);
#pragma unroll
        for (int d = 0; d < ND; d++) o[d] = f32x16{};
        m = -INFINITY;
        l = 0.f;
        r = kLeast;
        r_min = __builtin_bit_cast(float, kLeast << 23);
    }
    // X^T = K Q^T of the codes at lds + AT (JOINED), 32 dimensions a read, all reads first.
    template <int AT>
    __device__ __forceinline__ void scores8(const char* lds, f32x16 (&x)[NX]) {
        const int half = (threadIdx.x & 63) >> 5, row = threadIdx.x & 31;
        static_assert(NX == 1, "one run of 32 keys");
        constexpr int READS = NS / 2 < 4 ? NS / 2 : 4;
        u32x4 c[NS / 2];
        x[0] = f32x16{};
#pragma unroll
        for (int k = 0; k < NS / 2; k++) {
            const char* at = lds + row * DP + ((2 * k + half) ^ Place8<DP>::k(row)) * 16;
            c[k] = *reinterpret_cast<const u32x4*>(at + AT);
        }
#pragma unroll
        for (int k = 0; k < NS / 2; k++) {
            x[0] = mfma(halves(c[k][0], c[k][1]), qf[2 * k], x[0]);
            x[0] = mfma(halves(c[k][2], c[k][3]), qf[2 * k + 1], x[0]);
        }
        __builtin_amdgcn_sched_group_barrier(kDsRead, READS, 0);
#pragma unroll
        for (int k = 0; k < NS / 2; k++) {
            __builtin_amdgcn_sched_group_barrier(kValu, 20, 0);
            __builtin_amdgcn_sched_group_barrier(kMfma, 2, 0);
            if (k + READS < NS / 2) __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
        }
    }
    // Where in LDS this lane reads a tile of halves, formed once (the compiler would form
    // them again for every tile): of K chunk 2 k + half of key `lane & 31`, of V keys 8 w + 4
    // half .. + 3 of sixteen and dimensions 32 d .. + 31 by the transposing read.
    struct Places {
        uint32_t k[NS], v[ND][2];
        __device__ __forceinline__ explicit Places(const char* lds) {
            const uint32_t base = (uint32_t)(uintptr_t)(lmem*)lds;
            const int lane = threadIdx.x & 63, half = lane >> 5, row = lane & 31, g = lane >> 4 & 1, i = lane & 15;
#pragma unroll
            for (int c = 0; c < NS; c++) {
                k[c] = base + row * DP * 2 + ((2 * c + half) ^ Place16<DP>::k(row)) * 16;
                asm volatile("" : "+v"(k[c]));
            }
#pragma unroll
            for (int d = 0; d < ND; d++)
#pragma unroll
                for (int w = 0; w < 2; w++) {
                    const int key = 8 * w + 4 * half + (i >> 2), chunk = 4 * d + 2 * g + ((i & 3) >> 1);
                    v[d][w] = base + key * DP * 2 + (chunk ^ Place16<DP>::v(key)) * 16 + (i & 1) * 8;
                    asm volatile("" : "+v"(v[d][w]));
                }
        }
    };
    // The same of halves (not JOINED).  The reads run AHEAD of the products (one by one,
    // each waited for, they would be most of a tile's time).
    template <int AT>
    __device__ __forceinline__ void scores16(const Places& places, f32x16 (&x)[NX]) {
        constexpr int N = NX * NS, AHEAD = 6;
        f16x8 kf[N];
#pragma unroll
        for (int i = 0; i < N; i++) kf[i] = *(lmem16*)(uintptr_t)(places.k[i / NX] + (AT + 32 * (i % NX) * DP * 2));
#pragma unroll
        for (int n = 0; n < NX; n++) x[n] = f32x16{};
#pragma unroll
        for (int i = 0; i < N; i++) x[i % NX] = mfma(kf[i], qf[i / NX], x[i % NX]);
        __builtin_amdgcn_sched_group_barrier(kDsRead, AHEAD, 0);
#pragma unroll
        for (int i = 0; i < N - AHEAD; i++) {
            __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, AHEAD, 0);
    }
    // Scores with the keys' scales, and the running maximum and largest scale.  `there`
    // names the keys of the tile (from j0 on) that have a page, sc their scales: KT of keys,
    // then of values (sv: this lane's).  A half of the wave has sixteen of 32 keys, and each of its rows of
    // sixteen lanes holds their scales, one a lane, which the multiplication itself
    // broadcasts.  (Read from LDS for every lane they were a third of its traffic.)
    __device__ __forceinline__ void scaled(const AttnDev& a, const float* sc, int j0, unsigned long long there,
                                           f32x16 (&x)[NX], float (&sv)[NX]) {
        const int lane = threadIdx.x & 63, half = lane >> 5, mine = 8 * (lane >> 2 & 3) + 4 * half + (lane & 3);
        float sk[NX];
#pragma unroll
        for (int n = 0; n < NX; n++) {
            sk[n] = sc[32 * n + mine];
            sv[n] = sc[KT + 32 * n + mine];
        }
#pragma unroll
        for (int n = 0; n < NX; n++) times_lanes<0>(x[n], sk[n]);
        const unsigned long long all = KT == 64 ? ~0ull : (1ull << (KT & 63)) - 1;
        unsigned long long seen = ~0ull;
        if (!((there & all) == all && j0 + KT - 1 <= p_lo && (j0 >= z_hi || j0 + KT - 1 < a.sinks))) {
            if (a.scale == 0.f) {
#pragma unroll
                for (int n = 0; n < NX; n++) x[n] *= 0.f;
            }
            // the keys that this lane's row sees, from the first that the lane has on
            const auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
            seen = (there & below(p - j0 + 1) & (~below(z - j0) | below(a.sinks - j0))) >> (4 * half);
            const uint32_t word[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
            for (int n = 0; n < NX; n++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    x[n][e] = word[n] & (1u << (8 * (e / 4) + e % 4)) ? x[n][e] : -INFINITY;
        }
        float mt = max3(x[0][0], x[0][1], x[0][2]);
#pragma unroll
        for (int e = 3; e < 16 * NX - 1; e += 2) mt = max3(mt, x[e / 16][e % 16], x[(e + 1) / 16][(e + 1) % 16]);
        mt = max3(mt, mt, x[NX - 1][15]);
        mt = max_halves(mt) * c2;
        bool grows = mt > m + kSlack8;
#pragma unroll
        for (int n = 0; n < NX; n++) grows |= fabsf(sv[n]) > r_min;
        if (__any(grows)) {
            // (the largest scale that the row sees here; one that it does not see may be anything)
            const uint32_t word[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
            float st = 0.f;
#pragma unroll
            for (int n = 0; n < NX; n++) {
                f32x16 f;
#pragma unroll
                for (int e = 0; e < 16; e++) f[e] = word[n] & (1u << (8 * (e / 4) + e % 4)) ? 1.f : 0.f;
                // (0 * inf of an unseen scale is NaN, which the maximum passes over)
                times_lanes<1>(f, sv[n]);
#pragma unroll
                for (int e = 0; e < 16; e++) st = fmaxf(st, fabsf(f[e]));
            }
            st = max_halves(st);
            const int rn = min(max(r, (int)((__builtin_bit_cast(uint32_t, st) + 0x7fffffu) >> 23)), kMost);   // (up to a power of two)
            const float mn = fmaxf(m, mt);
            const float fix = (mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn)) *
                              __builtin_bit_cast(float, (127 + r - rn) << 23);
            l *= fix;
#pragma unroll
            for (int d = 0; d < ND; d++) o[d] *= fix;
            m = mn;
            r = rn;
            int least = r;
            for (int w = 32; w; w >>= 1) least = min(least, __shfl_xor(least, w));
            r_min = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(least) << 23);
        }
        mu = m == -INFINITY ? 0.f : m - kLift8 + (float)(r - 127);
    }
    // The weights of 32 keys.  (l takes them at once: one by one those below half of its
    // last bit would be lost, which a tail of 131071 keys at 2^-25 of the maximum is.)
    // `low` (or NULL): what the rounding to fp16 has left of each, as another fp16.
    __device__ __forceinline__ void form(f32x16& x, float sv, f16x8* pf, f16x8* low = nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e++) {
            x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], c2, -mu));
            sum += x[e];
        }
        times_lanes<2>(x, sv);
#pragma unroll
        for (int e = 0; e < 16; e++) pf[e / 8][e % 8] = (f16)x[e];
        if (low) {
#pragma unroll
            for (int e = 0; e < 16; e++) low[e / 8][e % 8] = (f16)(x[e] - (float)pf[e / 8][e % 8]);
        }
        l += sum;
    }
    // After the last tile: l with both halves' keys, and m as what a weight of 1 stands
    // for, by which parts are joined and lse is formed.
    __device__ __forceinline__ void finish() {
        l += __shfl_xor(l, 32);
        m += (float)(r - 127) - kLift8;
    }
    // This lane's part of a transposing read of codes: dimensions 32 d .. 32 d + 31,
    // sixteen keys.  Of 16 lanes, lane i names 8 bytes of key i / 2 (of eight) and gets
    // dimension i of all eight.  A half takes the keys whose weights it has: 4 half + 0 ..
    // 3 and 8 more.
    __device__ __forceinline__ static uint32_t v_part8(const char* lds, int d) {
        const int lane = threadIdx.x & 63, half = lane >> 5, g = (lane >> 4) & 1, i = lane & 15;
        const int key = 4 * half + (i >> 1 & 3) + 8 * (i >> 3);
        return (uint32_t)(uintptr_t)(lmem*)(lds + key * DP + ((2 * d + g) ^ Place8<DP>::v(key)) * 16 + (i & 1) * 8);
    }
    // O^T += V^T P^T of the codes at lds + AT, 16 keys a step.  Other tiles are on their
    // way to LDS meanwhile, and the compiler would wait for all of them before the reads'
    // builtin; so two steps of 128 dimensions are read, and waited for, at once.
    template <int AT, bool LOW>
    __device__ __forceinline__ void add8(const char* lds, const f16x8 (&pf)[2 * NX], const f16x8 (&low)[2 * NX]) {
        static_assert(AT + KT * DP <= 65536 && NX == 1, "offsets of a read");
        constexpr int W = ND < 4 ? 2 : 4;   // runs of 32 dimensions that are read at once
#pragma unroll
        for (int d = 0; d < ND; d += W) {
            u32x2 v[2][W];   // [step][dimensions]
            if constexpr (W == 2)
                asm volatile(
                    "ds_read_b64_tr_b8 %0, %4 offset:%6\n\tds_read_b64_tr_b8 %1, %5 offset:%6\n\t"
                    "ds_read_b64_tr_b8 %2, %4 offset:%7\n\tds_read_b64_tr_b8 %3, %5 offset:%7\n\t"
                    "s_waitcnt lgkmcnt(0)"
                    : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1])
                    : "v"(v_part8(lds, d)), "v"(v_part8(lds, d + 1)), "n"(AT), "n"(AT + 16 * DP)
                    : "memory");
            else
                asm volatile(
                    "ds_read_b64_tr_b8 %0, %8 offset:%12\n\tds_read_b64_tr_b8 %1, %9 offset:%12\n\t"
                    "ds_read_b64_tr_b8 %2, %10 offset:%12\n\tds_read_b64_tr_b8 %3, %11 offset:%12\n\t"
                    "ds_read_b64_tr_b8 %4, %8 offset:%13\n\tds_read_b64_tr_b8 %5, %9 offset:%13\n\t"
                    "ds_read_b64_tr_b8 %6, %10 offset:%13\n\tds_read_b64_tr_b8 %7, %11 offset:%13\n\t"
                    "s_waitcnt lgkmcnt(0)"
                    : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][W - 2]), "=&v"(v[0][W - 1]), "=&v"(v[1][0]), "=&v"(v[1][1]),
                      "=&v"(v[1][W - 2]), "=&v"(v[1][W - 1])
                    : "v"(v_part8(lds, d)), "v"(v_part8(lds, d + 1)), "v"(v_part8(lds, d + 2)), "v"(v_part8(lds, d + 3)),
                      "n"(AT), "n"(AT + 16 * DP)
                    : "memory");
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int c = 0; c < W; c++) {
                    const f16x8 f = halves(v[u][c][0], v[u][c][1]);
                    o[d + c] = mfma(f, pf[u], o[d + c]);
                    if constexpr (LOW) o[d + c] = mfma(f, low[u], o[d + c]);
                }
        }
    }
    // The weights of a tile (LOW: as two fp16 each) and O^T += V^T P^T of the halves at lds
    // + AT.  V's reads run ahead, and the weights of the second 32 keys are formed beside the
    // products of the first.
    template <int AT>
    __device__ __forceinline__ void read16(const Places& places, int u, f16x8 (&v)[ND]) {
#pragma unroll
        for (int d = 0; d < ND; d++) {
            union { s16x4 w[2]; f16x8 v; } f;
#pragma unroll
            for (int w = 0; w < 2; w++)
                f.w[w] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lmem4*)(uintptr_t)(places.v[d][w] + (AT + u * 16 * DP * 2)));
            v[d] = f.v;
        }
    }
    template <int AT, bool LOW>
    __device__ __forceinline__ void add16(const Places& places, f32x16 (&x)[NX], const float (&sv)[NX]) {
        f16x8 pf[2 * NX], low[2 * NX], v[2][ND];
        auto step = [&](int u) {
#pragma unroll
            for (int d = 0; d < ND; d++) {
                o[d] = mfma(v[u % 2][d], pf[u], o[d]);
                if constexpr (LOW) o[d] = mfma(v[u % 2][d], low[u], o[d]);
            }
        };
        read16<AT>(places, 0, v[0]);
        form(x[0], sv[0], pf, LOW ? low : nullptr);
        __builtin_amdgcn_sched_barrier(0);
        read16<AT>(places, 1, v[1]);
        step(0);
        if constexpr (NX == 2) {
            read16<AT>(places, 2, v[0]);
            step(1);
            form(x[1], sv[1], pf + 2, LOW ? low + 2 : nullptr);
#pragma unroll
            for (int i = 0; i < 2 * ND; i++) {
                __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 0);
                __builtin_amdgcn_sched_group_barrier(kMfma, LOW ? 2 : 1, 0);
                __builtin_amdgcn_sched_group_barrier(kValu, (LOW ? 112 : 80) / (2 * ND), 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            read16<AT>(places, 3, v[1]);
            step(2);
            step(3);
        } else {
            step(1);
        }
    }
};

// Where keys that are not there and dimensions past the head's come from.
__device__ const uint4 g_zeros8[QGEMV_HEAD_DIM_MAX / 16] = {};

// The pages of a tile's keys, from 64 columns of the table at a time (one a
// lane): a tile's columns are within 64 even with a page for every key.  A tile
// whose keys are all there, in pages of whole runs of 16 (a.runs), is addressed
// by scalars, one page and one offset a run, with products of 32 bits.  Any other
// has an offset for every key.
template <int DP, int KT>
struct Pages8 {
    static constexpr int CPR = DP / 16, RPI = 64 / CPR;   // chunks of a row; rows of a wave's load of 1 KB
    int first = -64, page = -1;            // the lane's column is first + lane
    unsigned long long valid = 0;          // columns with a page of the pool
    int j0;                                // the tile: its first key
    bool runs;                             // whether scalars do
    int64_t off, soff;                     // offsets of the codes and the scale of key `lane`, -1 where it is not there

    __device__ __forceinline__ void ask(const AttnDev& a, const int32_t* table) {
        const int lane = threadIdx.x & 63;
        first = 0;
        if (lane < a.ldt) page = table[lane];
    }
    __device__ __forceinline__ void arrive(const AttnDev& a) { valid = __ballot(page >= 0 && page < a.n_pages); }

    // Takes up the tile at key j; returns which of its keys are there.
    __device__ __forceinline__ unsigned long long tile(const Attn8Dev& a, const Span& s, const int32_t* table, int j) {
        const int lane = threadIdx.x & 63;
        j0 = j;
        off = soff = -1;
        const int c0 = a.page_shift >= 0 ? j0 >> a.page_shift : j0 / a.page_size;
        const int c1 = a.page_shift >= 0 ? (j0 + KT - 1) >> a.page_shift : (j0 + KT - 1) / a.page_size;
        if (c0 < first || c1 >= first + 64) {
            first = c0;
            page = first + lane < a.ldt ? table[first + lane] : -1;
            arrive(a);   // (the wait for the page is here, not at every tile)
        }
        const unsigned long long need = (2ull << (c1 - c0)) - 1;
        runs = a.runs && j0 + KT <= s.limit && (valid >> (c0 - first) & need) == need;
        if (__builtin_expect(runs, 1)) return ~0ull;
        const int key = j0 + (KT == 64 ? lane : lane & (KT - 1));
        const int c = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
        const int mine = __shfl(page, c - first);
        if (key < s.limit && mine >= 0 && mine < a.n_pages) {
            off = key_offset(a, mine, key);
            soff = scale_offset(a, mine, key);
        }
        return __ballot(off >= 0);
    }
    // Row `row` of the tile, the first or another of (part of) a run: its page, and where
    // it is.
    __device__ __forceinline__ uint32_t run_page(const AttnDev& a, int row) const {
        return __builtin_amdgcn_readlane(page, ((j0 + row) >> a.page_shift) - first);
    }
    __device__ __forceinline__ uint64_t run(const Attn8Dev& a, int row) const {
        return (uint64_t)run_page(a, row) * a.page_bytes + (uint32_t)((j0 + row) & (a.page_size - 1)) * a.slot_bytes;
    }
    // Where chunk `chunk` of the tile's row `row` is, of a tile that has no runs (of an
    // address, which may be nobody's, and `from`, the head's).
    __device__ __forceinline__ const char* single(const AttnDev& a, const char* from, int row, int chunk) const {
        const int64_t at = __shfl((long long)off, row);
        return at >= 0 && 16 * chunk < a.D ? from + at + 16 * chunk : (const char*)g_zeros8;
    }
    // Where the scale of the tile's row `row` is.
    __device__ __forceinline__ const float* scale(const Attn8Dev& a, const float* from, int row) const {
        if (__builtin_expect(runs, 1)) {
            uint32_t pg = run_page(a, 0);
#pragma unroll
            for (int u = 1; u < KT / 16; u++) pg = row >= 16 * u ? run_page(a, 16 * u) : pg;
            return from + ((uint64_t)pg * a.scale_page + (uint32_t)((j0 + row) & (a.page_size - 1)) * a.scale_slot);
        }
        const int64_t at = __shfl((long long)soff, row);
        return at >= 0 ? from + at : (const float*)g_zeros8;
    }
};

__device__ __forceinline__ void to_lds16(const void* from, char* to) {
    __builtin_amdgcn_global_load_lds((gmem*)from, (lmem*)to, 16, 0, 0);
}

// Many rows: NW waves of 32 rows each, which share every tile of KT keys.  The codes
// of the next tile are on their way to registers while one is used, and are made fp16
// once for all waves, on their way to LDS (by each wave for itself they would be 160
// vector instructions a tile, not 20 to 40).  Bound by the vector and the matrix pipe
// together, which hardly have their work at once: 289 and 32 instructions a wave and
// tile of 64 keys at 128 dimensions, busy 0.55 and 0.36 of the time at the 1.9 GHz that
// power leaves.  8192 tokens of 32 heads on 8, causal, take 640 to 650 us, 850 TFLOP/s
// (with the reads of K one by one and scales read from LDS for every lane 985).  Nine
// sequences of chunks of 64 dimensions take 58 us: 0.36 of a wave's time it waits for the tile
// that the step before sent for, vector pipe 0.48 busy.  Four waves at 128 dimensions take 715 us
// where eight take 645: they convert twice as much each.  With the first tile sent for
// before q is taken, 64 dimensions leave room for three workgroups a CU: a prompt of 4096
// of 14 heads on 2 takes 103 us, 122 without.
// 256 dimensions: one wave a SIMD, and a prompt of 4096 of 8 heads on 2 is one round of 256
// workgroups whose longest, 128 tiles of 1.8 us, is its 230 us.
template <typename T, typename TO, int DP, int KT, int NW, int OCC>
__global__ __launch_bounds__(64 * NW, OCC) void k_attn8_many(const Attn8Dev a) {
    typedef Rows8<DP, KT> R;
    constexpr int ROWS = 32 * NW, CPR = DP / 16, RPI = 64 / CPR;
    constexpr int TILE = KT * DP * 2, BUF = 2 * TILE;    // bytes of a K (or V) tile, and of both
    constexpr int LOADS = KT / RPI / NW;                 // wave loads of K (and of V) per wave
    constexpr int SC = 2 * KT;                           // scales of a tile
    // (one fp16 a weight, off by up to 2^-11, would be the whole error of an fp32 output: it takes
    // two, 2^-22.  Of fp16 outputs one leaves 2.9e-4 where their own rounding leaves 2.1e-4.  A
    // prompt of 8192, 32 heads on 8 of 128, takes 890 us so, 670 to 680 with one; 4096 tokens of
    // 14 on 2 of 64 136 and 96, of 8 on 2 of 256 261 and 230)
    constexpr bool LOW = std::is_same<TO, float>::value;
    static_assert(LOADS >= 1 && KT <= 64 && SC <= 64 * NW && SC % 64 == 0, "tile shape");
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    float* sc = reinterpret_cast<float*>(lds + 2 * BUF);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    // heads first, so that the workgroups of one head meet in one L2; the row
    // tiles with the most keys first
    const int h = blockIdx.x % a.heads;
    const int rest = blockIdx.x / a.heads;
    const int part = rest % a.splits, row_tile = a.row_tiles - 1 - rest / a.splits;
    const int b = blockIdx.y;
    const int32_t* table = a.table + b * a.ldt;
    Pages8<DP, KT> pages;
    pages.ask(a, table);
    Span s;
    if (!make_span<KT, ROWS>(a, b, row_tile, part, s)) return;

    // this lane's row, the last one of the block where it has none of its own
    const int first_row = row_tile * ROWS + 32 * wave, r = first_row + (lane & 31);
    const int r_end = (s.i1 + 1) * a.G;
    const int rc = min(r, r_end - 1);
    const bool active = first_row < r_end;
    R w;
    const auto query = w.template ask<T, false>(a, s, h, rc, first_row);
    pages.arrive(a);

    const char* kbase = (const char*)a.k + h * a.head_stride;
    const char* vbase = (const char*)a.v + h * a.head_stride;
    const float* sbase = (threadIdx.x < KT ? a.ks : a.vs) + h * a.scale_head_stride;
    u32x4 kc[LOADS], vc[LOADS];
    float scale;
    auto ask_tile = [&](int t) -> unsigned long long {
        const unsigned long long there = pages.tile(a, s, table, tile_of(s, t) * KT);
        constexpr int MINE = RPI * LOADS;    // rows of the tile that this wave takes, in one run
        static_assert(16 % MINE == 0, "rows of a wave");
        if (__builtin_expect(pages.runs, 1)) {
            const uint64_t run = pages.run(a, MINE * wave);
            const uint32_t at = (lane / CPR) * a.slot_bytes + 16 * (lane % CPR);
#pragma unroll
            for (int c = 0; c < LOADS; c++) {
                kc[c] = *(gmem16*)(kbase + run + (at + RPI * c * a.slot_bytes));
                vc[c] = *(gmem16*)(vbase + run + (at + RPI * c * a.slot_bytes));
            }
        } else {
#pragma unroll
            for (int c = 0; c < LOADS; c++) {
                const int row = MINE * wave + RPI * c + lane / CPR;
                kc[c] = *(gmem16*)pages.single(a, kbase, row, lane % CPR);
                vc[c] = *(gmem16*)pages.single(a, vbase, row, lane % CPR);
            }
        }
        if (wave < SC / 64) scale = *(gmemf*)pages.scale(a, sbase, threadIdx.x & (KT - 1));
        return there;
    };
    // (a row's chunk c of 16 codes becomes its chunks 2 c and 2 c + 1 of eight halves)
    auto put_tile = [&](int buf) {
        char* to = lds + buf * BUF;
#pragma unroll
        for (int c = 0; c < LOADS; c++) {
            const int row = RPI * (LOADS * wave + c) + lane / CPR, chunk = 2 * (lane % CPR);
            char* k = to + row * DP * 2;
            char* v = k + TILE;
            *reinterpret_cast<f16x8*>(k + (chunk ^ Place16<DP>::k(row)) * 16) = halves(kc[c][0], kc[c][1]);
            *reinterpret_cast<f16x8*>(k + (chunk + 1 ^ Place16<DP>::k(row)) * 16) = halves(kc[c][2], kc[c][3]);
            *reinterpret_cast<f16x8*>(v + (chunk ^ Place16<DP>::v(row)) * 16) = halves(vc[c][0], vc[c][1]);
            *reinterpret_cast<f16x8*>(v + (chunk + 1 ^ Place16<DP>::v(row)) * 16) = halves(vc[c][2], vc[c][3]);
        }
        if (wave < SC / 64) sc[buf * SC + threadIdx.x] = scale;
    };

    const typename R::Places places(lds);
    unsigned long long there = 0, there_next = 0;
    if (s.t0 < s.t1) {
        there = ask_tile(s.t0);
        w.start(a, query);
        put_tile(0);
    } else {
        w.start(a, query);
    }
    __syncthreads();
    auto step = [&](int t, auto buf) {
        constexpr int AT = buf * BUF;
        if (t + 1 < s.t1) there_next = ask_tile(t + 1);
        const int j0 = tile_of(s, t) * KT;
        if (active && j0 <= w.p_hi && (j0 + KT > w.z_lo || j0 < a.sinks)) {
            f32x16 x[R::NX];
            float sv[R::NX];
            w.template scores16<AT>(places, x);
            w.scaled(a, sc + buf * SC, j0, there, x, sv);
            w.template add16<AT + TILE, LOW>(places, x, sv);
        }
        if (t + 1 < s.t1) put_tile(1 - buf);
        __syncthreads();
        there = there_next;
    };
    for (int t = s.t0; t < s.t1; t += 2) {
        step(t, std::integral_constant<int, 0>{});
        if (t + 1 < s.t1) step(t + 1, std::integral_constant<int, 1>{});
    }
    if (!active) return;
    w.finish();

    bool bad = false;
#pragma unroll
    for (int d = 0; d < R::ND; d++)
#pragma unroll
        for (int e = 0; e < 16; e++) bad |= !(fabsf(w.o[d][e]) < INFINITY);
    bad |= !(fabsf(w.l) < INFINITY);
    bad |= __shfl_xor((int)bad, 32);
    const bool own = r < r_end;
    const int qi = rc / a.G, hq = h * a.G + rc - qi * a.G;
    const int64_t tok = s.s0 + qi, row = tok * a.q_heads + hq;
    if (own && !bad) {
        const int64_t at = row * a.splits + part;
        const float inv = s.parts > 1 ? 1.f : row_inverse(w.l);
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
        attn8_row<T, KT>(a, s, table, i, hh, a.scale * 1.4426950408889634f, ro, rm, rl);
        put_row<TO>(a, s, part, i, hh, ro, rm, rl);
    }
}

// At most 32 rows: each of NW waves takes a run of the tiles.  Its ring holds codes
// and scales of two tiles, straight from memory; a tile's K and scales make room for
// those after next as soon as the scores are formed, and V likewise, so that most
// of it is always on its way.  Codes become fp16 between LDS and the matrix cores.
// Bound by the way to memory: 64 sequences of up to 8192 keys, 32 heads on 8 of 128, take
// 186 to 189 us, 4.7 TB/s (the vector pipe is busy 0.4 of the time, the matrix cores 0.13).  Rows
// of 128 bytes a head, 1 KB apart, are part of that: with the heads' rows of a page
// together in memory the same takes 175.  Four waves and two workgroups a CU take 200,
// two or four heads a workgroup 188 to 196, more parts 211.
template <typename T, typename TO, int DP, int NW>
__global__ __launch_bounds__(64 * NW, (NW + 3) / 4) void k_attn8_few(const Attn8Dev a) {
    constexpr int KT = 32, ROWS = 32;
    typedef Rows8<DP, KT> R;
    // (the matrix cores have time to spare here, so that but for bf16, whose own rounding
    // is much the larger, weights are taken as two fp16 each)
    constexpr bool LOW = !std::is_same<TO, bf16>::value;
    constexpr int TILE = KT * DP, SCB = 2 * KT * 4, RING = 4 * TILE + 2 * SCB;   // K, K, V, V, scales, scales
    constexpr int CPR = DP / 16, RPI = 64 / CPR, LOADS = KT / RPI;             // wave loads of a tile
    extern __shared__ __attribute__((aligned(1024))) char lds[];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, row32 = lane & 31;
    // Workgroups go round the eight dies in turn.  A line of scales has a few keys of
    // several heads, so the heads of a part of a sequence run on one die and share it in
    // its L2 (the rule is at the launch).
    int h = blockIdx.x % a.heads, group = blockIdx.x / a.heads + a.splits * blockIdx.y;
    if (a.by_die) {
        h = blockIdx.x / 8;
        group = blockIdx.x % 8 + 8 * blockIdx.y;
    }
    const int b = group / a.splits, part = group - b * a.splits;
    if (b >= a.B) return;
    const int32_t* table = a.table + b * a.ldt;
    Pages8<DP, KT> pages;
    Span s;
    if (!make_span<KT, ROWS>(a, b, 0, part, s)) return;
    const int rows = (s.i1 + 1) * a.G;
    R w;
    const auto query = w.template ask<T, true>(a, s, h, min(row32, rows - 1), 0);

    const char* kbase = (const char*)a.k + h * a.head_stride;
    const char* vbase = (const char*)a.v + h * a.head_stride;
    const float* sbase = (half ? a.vs : a.ks) + h * a.scale_head_stride;
    char* mine = lds + wave * RING;
    const int each = (s.t1 - s.t0 + NW - 1) / NW;
    const int t0 = min(s.t0 + wave * each, s.t1), t1 = min(t0 + each, s.t1);
    auto take = [&](int t) { return pages.tile(a, s, table, tile_of(s, t) * KT); };
    // one wave load of 1 KB after another, a lane's chunk of a row by the chunk's place
    auto load = [&](const char* from, char* to, auto place) {
        if (__builtin_expect(pages.runs, 1)) {
            constexpr int PER = RPI < 16 ? 16 / RPI : 1;     // loads of a run
#pragma unroll
            for (int c = 0; c < LOADS; c++) {
                const char* base = from + pages.run(a, 16 * (c / PER));
                const int row = RPI * (c % PER) + lane / CPR;
                to_lds16(base + (row * a.slot_bytes + 16 * (lane % CPR ^ place(row))), to + 1024 * c);
            }
            return;
        }
#pragma unroll
        for (int c = 0; c < LOADS; c++) {
            const int row = RPI * c + lane / CPR;
            to_lds16(pages.single(a, from, row, lane % CPR ^ place(row)), to + 1024 * c);
        }
    };
    auto load_k = [&](int slot) {
        load(kbase, mine + slot * TILE, Place8<DP>::k);
        __builtin_amdgcn_global_load_lds((gmem*)pages.scale(a, sbase, row32), (lmem*)(mine + 4 * TILE + slot * SCB), 4, 0, 0);
    };
    auto load_v = [&](int slot) { load(vbase, mine + (2 + slot) * TILE, Place8<DP>::v); };
    if (t0 < t1) {
        unsigned long long there[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (t0 + i >= t1) break;
            there[i] = take(t0 + i);
            load_k(i);
            load_v(i);
        }
        w.start(a, query);
        auto step = [&](int t, auto at) {
            constexpr int SLOT = at;
            f32x16 x[R::NX];
            float sv[R::NX];
            // (loads land in their order: K S V of this tile, K S V of the next, K S of the one after)
            const int left = t1 - 1 - t;
            if (left > 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * LOADS + 1) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
            w.template scores8<SLOT * TILE>(mine, x);
            w.scaled(a, reinterpret_cast<const float*>(mine + 4 * TILE + SLOT * SCB), tile_of(s, t) * KT, there[0], x, sv);
            QGEMV_WAIT("lgkmcnt(0)");
            there[0] = there[1];
            if (left > 1) {
                there[1] = take(t + 2);
                load_k(SLOT);
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * LOADS + 2) : "memory");
            } else if (left > 0) {
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LOADS + 1) : "memory");
            } else {
                QGEMV_WAIT("vmcnt(0)");
            }
            f16x8 pf[2], low[2];
            w.form(x[0], sv[0], pf, LOW ? low : nullptr);
            w.template add8<(2 + SLOT) * TILE, LOW>(mine, pf, low);
            QGEMV_WAIT("lgkmcnt(0)");
            if (left > 1) load_v(SLOT);
        };
        for (int t = t0; t < t1; t += 2) {
            step(t, std::integral_constant<int, 0>{});
            if (t + 1 < t1) step(t + 1, std::integral_constant<int, 1>{});
        }
        w.finish();
    } else {
        w.start(a, query);
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
        bool bad = !(fabsf(sum) < INFINITY);
#pragma unroll
        for (int c = 0; c < DP / 64; c++) bad |= !(fabsf(f[c]) < INFINITY);
        const int i = rr / a.G, hh = h * a.G + rr - i * a.G;
        if (__any(bad))
            attn8_row<T, KT>(a, s, table, i, hh, a.scale * 1.4426950408889634f, f, top, sum);
        put_row<TO>(a, s, part, i, hh, f, top, sum);
    }
}

// (The rule and its places are those of the attention over 16 bits, though a CU holds three
// workgroups of 64 dimensions here, two with an fp32 output.  Over 14 sizes of 300 to 4096
// queries 768 places for 512 and for 1024 took 0.96 of the time, 0.81 to 1.12 (2 x 2000 queries over
// 4000 keys, 14 heads on 2, 125 us and 102; 4 x 300 over 8192, 16 on 16, 81 and 90), and with fp32
// out 1.00, 0.78 to 1.27.)
template <typename T, typename TO, int DP, int KT, int OCC, int NW>
static void launch_many(Attn8Dev d, const Attn8Args& a, hipStream_t st) {
    constexpr int ROWS = 32 * NW;
    split(d, a.max_kv, ROWS, KT, 4, 256 * OCC * 4 / NW, DP == 64 ? 1024 : 0, a.ws_bytes, a.ws);
    launch_kernel(k_attn8_many<T, TO, DP, KT, NW, OCC>,
                  dim3((unsigned)(d.heads * d.splits * d.row_tiles), (unsigned)d.B), dim3(64 * NW),
                  2 * (2 * KT * DP * 2 + 2 * KT * 4), st, d);
    join<TO, KT, ROWS, DP / 4>(d, st);
}
template <typename T, typename TO, int DP, int NW>
static void launch_few(Attn8Dev d, const Attn8Args& a, hipStream_t st) {
    split(d, a.max_kv, 32, 32, 4 * NW, 256, 0, a.ws_bytes, a.ws);
    // The heads of a part on one die, or each where its turn comes.  64 sequences of 8192 keys, 32
    // heads on 8 of 80: 182 and 247 us, of 128 187 and 198, 14 on 2 of 64 38 and 47.  A die then has
    // up to `heads` workgroups more than another, and 32 CUs (two workgroups each at 64 dimensions):
    // with up to 16 cache heads, over 66 sizes of 9 to 100 parts of up to 3000 keys, one die took
    // 0.74 to 1.05 of the time, 0.94 in the mean.  With 20 to 64 it took up to 1.6 where some dies
    // have a part more (9 parts of 32 on 32 of 128: 67 and 42 us; 33: 166 and 143), and 0.84 to 1.06
    // where they have a ninth more at the most (65 and 100 parts).  With fewer than eight parts
    // dies would be left without work (6 of 4096 keys, 32 on 32 of 128: 56 and 55 us).
    const int64_t groups = (int64_t)d.B * d.splits, dealt = (groups + 7) / 8 * 8;
    d.by_die = groups >= 8 && (d.heads <= 16 || 9 * dealt < 10 * groups);
    launch_kernel(k_attn8_few<T, TO, DP, NW>,
                  d.by_die ? dim3(8u * d.heads, (unsigned)((groups + 7) / 8)) : dim3((unsigned)(d.heads * d.splits), (unsigned)d.B),
                  dim3(64 * NW), NW * (4 * 32 * DP + 512 + 256), st, d);
    join<TO, 32, 32, DP / 4>(d, st);
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
    constexpr int64_t k31 = (int64_t)1 << 31;
    d.runs = (d.D == 64 || d.D == 128 || d.D == 256) && d.page_shift >= 4 && d.page_stride < k31 &&
             d.scale_page_stride < k31 && d.token_stride < k31 && d.token_stride * d.page_size < k31 &&
             d.scale_token_stride < k31 && d.scale_token_stride * d.page_size < k31;
    d.page_bytes = (uint32_t)d.page_stride; d.slot_bytes = (uint32_t)d.token_stride;
    d.scale_page = (uint32_t)d.scale_page_stride; d.scale_slot = (uint32_t)d.scale_token_stride;
    // (by the most queries of the call: single tokens beside a chunk go with the chunk, 63 over up
    // to 8192 keys beside 512 queries over 2000, 32 heads on 8 of 128, 1469 us, 246 in two calls)
    const bool few = (int64_t)a.max_q * d.G <= 32;
    with_type16(a.q_type, [&](auto t) {
        with_type(a.out_type, [&](auto to) {
            using T = decltype(t);
            using TO = decltype(to);
            if (few) {
                if (d.D <= 64) launch_few<T, TO, 64, 8>(d, a, st);
                else if (d.D <= 128) launch_few<T, TO, 128, 8>(d, a, st);
                else launch_few<T, TO, 256, 4>(d, a, st);
            } else {
                if (d.D <= 64) launch_many<T, TO, 64, 64, 2, 4>(d, a, st);
                else if (d.D <= 128) launch_many<T, TO, 128, 64, 2, 8>(d, a, st);
                else launch_many<T, TO, 256, 32, 1, 4>(d, a, st);
            }
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
