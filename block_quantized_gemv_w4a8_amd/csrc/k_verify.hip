// k_verify.hip -- verification of drafted tokens against the target's
// probabilities, and the token that follows the accepted ones.
//
// With x the logits of a row, M their largest and t the temperature, p(v) = e(v) /
// S, e(v) = exp((x_v - M) / t), S = sum e.  Draft i is accepted if u q(token) <
// p(token); the next token is the first v whose running sum of weights (p, or max(p
// - q, 0) behind a refused draft) passes u times the sum of all.  Such a border lies
// between two of V running sums, so a sum that is off by a share d moves about V d
// of the draws; with 2^-24 that would be one in a hundred of a flat row of 128256,
// hence 64 bits for exponentials and sums.
//
// A row is taken in chunks of 1024 values, a wave each, with its own largest value
// and sum (joined with exp((m - M) / t)), so that sums over chunks give the chunk in
// which the border lies and only that one is walked value by value.
//
// Three launches: the chunks of all rows; for each sequence what is accepted (found
// again by every workgroup: a few loads) and the sums of what a refused draft leaves of
// each chunk; the draw.  Certain drafts leave the chunks' own sums but for one, so the
// second goes into the third.  (With the draw left to the workgroup that comes last, the
// releases of memory that this takes made the second launch 31 us of 84.)  48 sequences
// of up to five rows of 128256 fp32 logits take 48 to 51 us: 29.5, 12.5 and 6.  The first
// is bound by the vector pipe (0.82 busy, 28 instructions a value of which 17 are the
// exponential and its sum; the bytes take 3.8 TB/s), the others by the way through stats,
// logits and sums.
#include <algorithm>

#include "qgemv_layer.h"

namespace qgemv {

constexpr int VWG = 256;           // threads of a workgroup
constexpr int VWAVES = VWG / 64;
constexpr int VPL = 16;            // values of a chunk a lane
constexpr int VCH = 64 * VPL;      // values of a chunk

// A chunk of a row: sum of e against its own largest value, which is first at `at`
// (looked for only where the temperature is 0).
struct ChunkStat {
    double sum;
    float top;
    int at;
};

// What a row's chunks say together: its largest value, first at `best`, and the sum.
struct RowStat {
    double inv;      // 1 / sum, 0 where there is no mass
    float top;
    int best;
};
// What the second launch found of a sequence: the row that the next token comes from,
// `done` rows on.
struct Choice {
    RowStat row;
    int done;
};

struct VerifyDev {
    const void* logits;
    const int32_t *q_start, *tokens;
    const float *draft, *u, *temperature;
    int32_t *accepted, *next;
    ChunkStat* stats;     // [B][max_q][chunks]
    double* left;         // [B][chunks]
    Choice* choice;       // [B]
    int64_t ldl, ldd;
    int T, V, B, max_q, chunks;
};

// 2^z for z <= 0 (0 for NaN): 2^f, |f| <= 1/2 what is left of z beside a whole number n,
// as 1 + f g(f) with g of degree 8 interpolated at Chebyshev's points (off by 4e-14, exact
// at 0).  The coefficients are kept in registers (of scalars each step would copy one
// first).
struct Series {
    double c[9];
    __device__ __forceinline__ Series() {
        constexpr double g[9] = {0.6931471805599453, 0.2402265069581299, 0.055504108664760424, 0.009618129159402558,
                                 0.0013333558179043112, 0.00015403455852453838, 1.525268684626772e-05, 1.3255224878668817e-06,
                                 1.0203121063391729e-07};
#pragma unroll
        for (int i = 0; i < 9; i++) {
            c[i] = g[i];
            asm volatile("" : "+v"(c[i]));
        }
    }
    __device__ __forceinline__ double part(double f) const {
        double p = c[8];
#pragma unroll
        for (int i = 7; i >= 0; i--) p = fma(p, f, c[i]);
        return fma(p, f, 1.0);
    }
    __device__ __forceinline__ double power(double z) const {
        z = fmax(z, -1100.0);
        const double n = rint(z);
        return ldexp(part(z - n), (int)n);
    }
    // The same but for 2^-1000 where that is less: n is left in the low bits of a sum, and
    // added to the exponent.  (For sums over a row, whose largest is 1: instructions of the
    // full rate only.)
    __device__ __forceinline__ double above(double z) const {
        constexpr double kWhole = 6755399441055744.0;   // 1.5 * 2^52
        z = fmax(z, -1000.0);
        const double t = z + kWhole;
        const double p = part(z - (t - kWhole));
        return __hiloint2double(__double2hiint(p) + (__double2loint(t) << 20), __double2loint(p));
    }
};

// The rows of sequence b, and its temperature.
struct Seq {
    int s0, n;
    bool greedy;
    double inv;      // log2(e) / temperature
    Series series;
};
__device__ __forceinline__ Seq sequence(const VerifyDev& a, int b) {
    Seq s;
    s.s0 = min(max(a.q_start[b], 0), a.T);
    s.n = min(min(max(a.q_start[b + 1], s.s0), a.T) - s.s0, a.max_q);
    const float t = a.temperature ? a.temperature[b] : 1.f;
    s.greedy = !(t > 0.f);
    s.inv = 1.4426950408889634 / (double)t;
    return s;
}

// e of a logit against the largest, top (not -inf): a -inf has none whatever the
// temperature (-inf * 0 is NaN).
__device__ __forceinline__ double mass(float x, float top, const Seq& s) { return s.series.power(((double)x - (double)top) * s.inv); }
// A logit as it counts: -inf for NaN, the largest number for +inf.
__device__ __forceinline__ float real(float x) { return x == x ? fminf(x, 3.402823466e38f) : -INFINITY; }
template <typename T>
__device__ __forceinline__ float logit(const T* row, int v) {
    return real((float)row[v]);
}

// Sixteen values of chunk c of a row, -inf past its end; value i of lane l is
// number place<T>(c, i) of the row.  (Rows need no alignment beyond their elements'.)
template <typename T>
__device__ __forceinline__ int place(int c, int i) {
    constexpr int G = 16 / sizeof(T);
    return c * VCH + i / G * (64 * G) + (threadIdx.x & 63) * G + i % G;
}
template <typename T>
__device__ __forceinline__ void chunk_values(const T* row, int V, int c, float (&x)[VPL]) {
    constexpr int G = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < VPL; i += G) {
        const int v = place<T>(c, i);
        T e[G];
        if (v + G <= V) {
            __builtin_memcpy(e, row + v, sizeof e);
#pragma unroll
            for (int j = 0; j < G; j++) x[i + j] = (float)e[j];
        } else {
#pragma unroll
            for (int j = 0; j < G; j++) x[i + j] = v + j < V ? (float)row[v + j] : -INFINITY;
        }
    }
}

template <typename X, typename F>
__device__ __forceinline__ X over_wave(X x, F f) {
    for (int w = 32; w; w >>= 1) x = f(x, __shfl_xor(x, w));
    return x;
}
__device__ __forceinline__ double wave_sum(double x) {
    return over_wave(x, [](double p, double q) { return p + q; });
}
__device__ __forceinline__ float wave_max(float x) {
    return over_wave(x, [](float p, float q) { return fmaxf(p, q); });
}
__device__ __forceinline__ int wave_min(int x) {
    return over_wave(x, [](int p, int q) { return min(p, q); });
}

// One chunk of a row, by a wave that has its values.
template <typename T>
__device__ __forceinline__ ChunkStat chunk_stat(float (&x)[VPL], int c, const Seq& s) {
    // (the maximum passes over NaN, and above() takes a NaN as the least)
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; i++) top = fmaxf(top, x[i]);
    top = wave_max(top);
    if (top == INFINITY) {
        top = real(top);
#pragma unroll
        for (int i = 0; i < VPL; i++) x[i] = real(x[i]);
    }
    ChunkStat r{0.0, top, 0};
    if (top == -INFINITY) return r;
    if (s.greedy) {
        int at = INT32_MAX;
#pragma unroll
        for (int i = VPL - 1; i >= 0; i--) at = x[i] == top ? place<T>(c, i) : at;
        r.at = wave_min(at);
        return r;
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; i++) sum += s.series.above(((double)x[i] - (double)top) * s.inv);
    r.sum = wave_sum(sum);
    return r;
}

__device__ __forceinline__ double chunk_mass(const ChunkStat& c, float top, const Seq& s) {
    return c.sum > 0.0 ? c.sum * mass(c.top, top, s) : 0.0;
}
// (by a wave, which has up to HELD chunks a lane at hand and reads the others twice)
__device__ RowStat row_stat(const ChunkStat* stats, int chunks, const Seq& s) {
    constexpr int HELD = 3;
    const int lane = threadIdx.x & 63;
    ChunkStat held[HELD];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < HELD; i++) {
        held[i] = ChunkStat{0.0, -INFINITY, 0};
        if (lane + 64 * i < chunks) held[i] = stats[lane + 64 * i];
    }
#pragma unroll
    for (int i = 0; i < HELD; i++) top = fmaxf(top, held[i].top);
    for (int c = lane + 64 * HELD; c < chunks; c += 64) top = fmaxf(top, stats[c].top);
    top = wave_max(top);
    RowStat r{0.0, top, -1};
    if (top == -INFINITY) return r;
    if (s.greedy) {
        int at = INT32_MAX;
#pragma unroll
        for (int i = 0; i < HELD; i++)
            if (held[i].top == top) at = min(at, held[i].at);
        for (int c = lane + 64 * HELD; c < chunks; c += 64)
            if (stats[c].top == top) at = min(at, stats[c].at);
        r.best = wave_min(at);
        return r;
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < HELD; i++) sum += chunk_mass(held[i], top, s);
    for (int c = lane + 64 * HELD; c < chunks; c += 64) sum += chunk_mass(stats[c], top, s);
    r.inv = 1.0 / wave_sum(sum);
    return r;
}
// p of a logit.
__device__ __forceinline__ double prob(float x, const RowStat& r, const Seq& s) { return mass(x, r.top, s) * r.inv; }

// What the acceptance of the draft behind a row takes, asked for ahead of the row's sum.
struct Draft {
    int token;     // -1: none that can be accepted
    float x, q, u;
};
template <typename T>
__device__ __forceinline__ Draft draft_of(const VerifyDev& a, int row) {
    Draft d{a.tokens[row + 1], 0.f, 1.f, a.u[row + 1]};
    if (d.token < 0 || d.token >= a.V) d.token = -1;
    if (d.token < 0) return d;
    d.x = logit((const T*)a.logits + (int64_t)row * a.ldl, d.token);
    if (a.draft) d.q = a.draft[(int64_t)(row + 1) * a.ldd + d.token];
    return d;
}
__device__ __forceinline__ bool passes(const Draft& d, const RowStat& r, const Seq& s) {
    if (d.token < 0 || r.top == -INFINITY) return false;
    const double p = s.greedy ? (d.token == r.best ? 1.0 : 0.0) : prob(d.x, r, s);
    return (double)d.u * (d.q > 0.f ? (double)d.q : 0.0) < p;
}

// The weights that the next token is drawn by: p, or what the draft leaves of it.
enum Kind { kWhole, kLeft };
__device__ __forceinline__ double weight(const VerifyDev& a, Kind kind, int row, int v, float x, float q, const RowStat& r, const Seq& s) {
    const double p = prob(real(x), r, s);
    if (kind == kWhole) return p;
    if (!a.draft) return v == a.tokens[row + 1] ? 0.0 : p;
    const double w = p - (q > 0.f ? (double)q : 0.0);
    return w > 0.0 ? w : 0.0;
}
// The sum of what a draft leaves of a chunk, by a wave, of a row that has mass.
template <typename T>
__device__ double chunk_left(const VerifyDev& a, int row, int c, const RowStat& r, const Seq& s) {
    float x[VPL], q[VPL] = {};
    chunk_values((const T*)a.logits + (int64_t)row * a.ldl, a.V, c, x);
    if (a.draft) {
        // (at the places of x)
        constexpr int G = 16 / sizeof(T);
        const float* d = a.draft + (int64_t)(row + 1) * a.ldd;
#pragma unroll
        for (int i = 0; i < VPL; i += G) {
            const int v = place<T>(c, i);
            if (v + G <= a.V) __builtin_memcpy(q + i, d + v, sizeof(float) * G);
            else
                for (int j = 0; j < G; j++) q[i + j] = v + j < a.V ? d[v + j] : 0.f;
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; i++) sum += weight(a, kLeft, row, place<T>(c, i), x[i], q[i], r, s);
    return wave_sum(sum);
}

// The sum of x over the threads before this one, and over all.
__device__ double before(double x, double& total, double* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double sum = x;
    for (int w = 1; w < 64; w <<= 1) {
        const double y = __shfl_up(sum, w);
        if (lane >= w) sum += y;
    }
    __syncthreads();
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    double head = 0.0;
    total = 0.0;
#pragma unroll
    for (int w = 0; w < VWAVES; w++) {
        if (w < wave) head += part[w];
        total += part[w];
    }
    return head + sum - x;
}
// The smallest of the threads' numbers.
__device__ int least(int x, int* part) {
    x = wave_min(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    return min(min(part[0], part[1]), min(part[2], part[3]));
}

// The token that is drawn, by the workgroup, from the weights of a row whose chunks'
// sums are sum(c); -1 if they are all 0.
template <typename T, typename S>
__device__ int drawn(const VerifyDev& a, Kind kind, int row, float u, const RowStat& r, const Seq& s, S sums) {
    __shared__ double part[VWAVES], start;
    __shared__ int ipart[VWAVES];
    const int each = (a.chunks + VWG - 1) / VWG, c0 = threadIdx.x * each, c1 = min(c0 + each, a.chunks);
    double own = 0.0, total;
    for (int c = c0; c < c1; c++) own += sums(c);
    double run = before(own, total, part);
    if (!(total > 0.0)) return -1;
    const double aim = u > 0.f ? (double)u * total : 0.0;
    int found = INT32_MAX, last = INT32_MAX;     // (last: counted from the end)
    double base = 0.0;
    for (int c = c0; c < c1; c++) {
        const double w = sums(c);
        if (w > 0.0) last = a.chunks - 1 - c;
        // (a thread's first sum may be a last bit above what the thread before it ends with: a
        // chunk without weight would then pass for the border's)
        if (found == INT32_MAX && w > 0.0 && run + w > aim) {
            found = c;
            base = run;
        }
        run += w;
    }
    const int first = least(found, ipart);
    const int end = a.chunks - 1 - least(last, ipart);
    const bool none = first == INT32_MAX;
    const int c = none ? end : first;
    if (!none && found == first) start = base;
    __syncthreads();
    const double from = none ? 0.0 : start;
    // value by value: each thread has four of them
    constexpr int EACH = VCH / VWG;
    const T* x = (const T*)a.logits + (int64_t)row * a.ldl;
    const float* q = a.draft ? a.draft + (int64_t)(row + 1) * a.ldd : nullptr;
    double w[EACH];
    own = 0.0;
#pragma unroll
    for (int i = 0; i < EACH; i++) {
        const int v = c * VCH + EACH * (int)threadIdx.x + i;
        w[i] = v < a.V ? weight(a, kind, row, v, (float)x[v], kind == kLeft && q ? q[v] : 0.f, r, s) : 0.0;
        own += w[i];
    }
    double chunk;
    run = from + before(own, chunk, part);
    found = last = INT32_MAX;
#pragma unroll
    for (int i = 0; i < EACH; i++) {
        const int v = EACH * (int)threadIdx.x + i;
        run += w[i];
        if (w[i] > 0.0) last = VCH - 1 - v;
        if (!none && found == INT32_MAX && run > aim && w[i] > 0.0) found = v;
    }
    const int at = least(found, ipart), tail = least(last, ipart);
    return c * VCH + (at != INT32_MAX ? at : tail != INT32_MAX ? VCH - 1 - tail : 0);
}
// The token after the accepted ones where no sums of what is left are at hand: from
// the chunks of the row itself, with the chunk of a certain token that was refused
// summed without it.
template <typename T>
__device__ int drawn_whole(const VerifyDev& a, bool refused, int row, float u, const RowStat& r, const Seq& s, const ChunkStat* stats) {
    __shared__ double rest;
    if (!(r.inv > 0.0)) return -1;
    // (by p of the chunk's largest: where that is 0 its tokens weigh nothing one by one either,
    // while a sum of their exponentials may still hold a bit)
    const auto whole = [&](int c) {
        const ChunkStat k = stats[c];
        return k.sum > 0.0 ? k.sum * prob(k.top, r, s) : 0.0;
    };
    if (refused && !a.draft) {
        const int token = a.tokens[row + 1], its = token >= 0 && token < a.V ? token / VCH : -1;
        if (threadIdx.x < 64 && its >= 0) {
            const double w = chunk_left<T>(a, row, its, r, s);
            if (threadIdx.x == 0) rest = w;
        }
        __syncthreads();
        const int next = drawn<T>(a, kLeft, row, u, r, s, [&](int c) { return c == its ? rest : whole(c); });
        if (next >= 0) return next;
    }
    return drawn<T>(a, kWhole, row, u, r, s, whole);
}

// The chunks of all rows, one a wave.
template <typename T>
__global__ __launch_bounds__(VWG) void k_verify_stats(const VerifyDev a) {
    const int c = blockIdx.x * VWAVES + (threadIdx.x >> 6), i = blockIdx.y, b = blockIdx.z;
    const Seq s = sequence(a, b);
    if (i >= s.n || c >= a.chunks) return;
    float x[VPL];
    chunk_values((const T*)a.logits + (int64_t)(s.s0 + i) * a.ldl, a.V, c, x);
    const ChunkStat r = chunk_stat<T>(x, c, s);
    if ((threadIdx.x & 63) == 0) a.stats[((int64_t)b * a.max_q + i) * a.chunks + c] = r;
}

// What is accepted of a sequence, by a workgroup, for all its threads: the first row
// whose draft is refused, four rows at a time (the last row has none).
template <typename T>
__device__ Choice choose(const VerifyDev& a, int b, const Seq& s) {
    __shared__ int stop;
    __shared__ RowStat at;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const ChunkStat* stats = a.stats + (int64_t)b * a.max_q * a.chunks;
    if (threadIdx.x == 0) {
        stop = s.n > 0 ? s.n - 1 : 0;
        at = RowStat{0.0, -INFINITY, -1};
    }
    __syncthreads();
    for (int i0 = 0; i0 < s.n; i0 += VWAVES) {
        const int i = i0 + wave;
        RowStat r{};
        bool ends = false;
        if (i < s.n) {
            Draft d{};
            if (i + 1 < s.n) d = draft_of<T>(a, s.s0 + i);
            r = row_stat(stats + (int64_t)i * a.chunks, a.chunks, s);
            ends = i + 1 == s.n || !passes(d, r, s);
        }
        if (ends && lane == 0) atomicMin(&stop, i);
        __syncthreads();
        const int now = stop;
        if (ends && i == now && lane == 0) at = r;
        __syncthreads();
        if (now < i0 + VWAVES) break;
    }
    return Choice{at, stop};
}

// What is accepted, and the sums of what a refused draft leaves of each chunk, PER chunks a wave.
template <typename T, int PER>
__global__ __launch_bounds__(VWG) void k_verify_left(const VerifyDev a) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, b = blockIdx.y;
    const Seq s = sequence(a, b);
    const Choice pick = choose<T>(a, b, s);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.choice[b] = pick;
    if (s.n == 0 || s.greedy || pick.done + 1 >= s.n || !(pick.row.inv > 0.0)) return;
    const int c0 = (blockIdx.x * VWAVES + wave) * PER;
    for (int c = c0; c < min(c0 + PER, a.chunks); c++) {
        const double w = chunk_left<T>(a, s.s0 + pick.done, c, pick.row, s);
        if (lane == 0) a.left[(int64_t)b * a.chunks + c] = w;
    }
}

// The next token; where drafts are certain, what is accepted too.
template <typename T, bool CERTAIN>
__global__ __launch_bounds__(VWG) void k_verify_draw(const VerifyDev a) {
    const int b = blockIdx.x;
    const Seq s = sequence(a, b);
    Choice pick;
    if constexpr (CERTAIN) pick = choose<T>(a, b, s);
    else pick = a.choice[b];
    const int row = s.s0 + pick.done;
    const bool refused = pick.done + 1 < s.n;
    int next = -1;
    if (s.n > 0 && s.greedy) {
        next = pick.row.best;
    } else if (s.n > 0 && pick.row.inv > 0.0) {
        const float u = a.u[s.s0];
        if (refused && !CERTAIN) {
            const double* left = a.left + (int64_t)b * a.chunks;
            next = drawn<T>(a, kLeft, row, u, pick.row, s, [&](int c) { return left[c]; });
        }
        if (next < 0)
            next = drawn_whole<T>(a, refused, row, u, pick.row, s, a.stats + ((int64_t)b * a.max_q + pick.done) * a.chunks);
    }
    if (threadIdx.x == 0) {
        a.accepted[b] = pick.done;
        a.next[b] = next;
    }
}

// A sequence by one workgroup, row by row.
template <typename T>
__global__ __launch_bounds__(VWG) void k_verify_one(const VerifyDev a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    ChunkStat* stats = reinterpret_cast<ChunkStat*>(lds);
    double* sums = reinterpret_cast<double*>(lds + (size_t)a.chunks * sizeof(ChunkStat));
    const int b = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Seq s = sequence(a, b);
    int done = 0, next = -1;
    for (int i = 0; i < s.n; i++) {
        const int row = s.s0 + i;
        __syncthreads();
        for (int c = wave; c < a.chunks; c += VWAVES) {
            float x[VPL];
            chunk_values((const T*)a.logits + (int64_t)row * a.ldl, a.V, c, x);
            const ChunkStat st = chunk_stat<T>(x, c, s);
            if (lane == 0) stats[c] = st;
        }
        __syncthreads();
        const RowStat r = row_stat(stats, a.chunks, s);
        const bool refused = i + 1 < s.n;
        if (refused && passes(draft_of<T>(a, row), r, s)) {
            done++;
            continue;
        }
        if (s.greedy) {
            next = r.best;
            break;
        }
        const float u = a.u[s.s0];
        if (refused && a.draft && r.inv > 0.0) {
            for (int c = wave; c < a.chunks; c += VWAVES) {
                const double w = chunk_left<T>(a, row, c, r, s);
                if (lane == 0) sums[c] = w;
            }
            __syncthreads();
            next = drawn<T>(a, kLeft, row, u, r, s, [&](int c) { return sums[c]; });
        }
        if (next < 0) next = drawn_whole<T>(a, refused, row, u, r, s, stats);
        break;
    }
    if (threadIdx.x == 0) {
        a.accepted[b] = done;
        a.next[b] = next;
    }
}

hipError_t launch_verify_draft(const VerifyArgs& a, hipStream_t st) {
    VerifyDev d{};
    d.logits = a.logits; d.q_start = a.q_start; d.tokens = a.tokens; d.draft = a.draft; d.u = a.u;
    d.temperature = a.temperature; d.accepted = a.accepted; d.next = a.next;
    d.ldl = a.ldl; d.ldd = a.ldd;
    d.T = (int)a.T; d.V = (int)a.V; d.B = a.B; d.max_q = a.max_q;
    d.chunks = (int)((a.V + VCH - 1) / VCH);
    // the workspace: what is chosen of each sequence, what drafts leave of each chunk, and
    // the chunks of all rows
    const int64_t choice = ((int64_t)d.B * sizeof(Choice) + 15) / 16 * 16, left = ((int64_t)d.B * d.chunks * 8 + 15) / 16 * 16;
    const int64_t rows = (int64_t)d.B * d.max_q;
    const int64_t most = std::min<int64_t>(a.ws_bytes, QGEMV_WS_BYTES);
    const bool fits = rows > 0 && choice + left <= most && rows <= (most - choice - left) / (d.chunks * (int64_t)sizeof(ChunkStat));
    d.choice = (Choice*)a.ws;
    d.left = (double*)((char*)a.ws + choice);
    d.stats = (ChunkStat*)((char*)a.ws + choice + left);
    with_type(a.logits_type, [&](auto t) {
        using T = decltype(t);
        // (few chunks of few sequences: one workgroup each.  With probabilities, against three launches:
        // 4 rows of 2000 values 11.3 us and 13.1, of 4096 11.9 and 13.0, of 6000 20.7 and 11.9; 4 sequences
        // of 2 rows of 4096 10.1 and 12.7, of 4 14.2 and 13.7, 8 of 4 15.4 and 15.0.  Certain drafts,
        // against two: 1 row of 600 7.4 and 9.2, 4 of 2000 10.0 and 11.5, of 4096 9.9 and 11.4, of 6000 20.7
        // and 10.2; 4 sequences of 2 rows of 4096 10.1 and 11.6, of 4 12.0 and 11.8, 8 of 4 12.9 and 11.9)
        if (fits && ((int64_t)d.chunks * d.max_q > 16 || d.B > 4)) {
            const auto groups = [&](int per) { return (unsigned)((d.chunks + VWAVES * per - 1) / (VWAVES * per)); };
            launch_kernel(k_verify_stats<T>, dim3(groups(1), (unsigned)d.max_q, (unsigned)d.B), dim3(VWG), 0, st, d);
            if (!d.draft) {
                launch_kernel(k_verify_draw<T, true>, dim3((unsigned)d.B), dim3(VWG), 0, st, d);
                return;
            }
            // (chunks a wave: 9072 in all, 72 sequences of 126, take 39 us by one and 41 by four, 12800 47
            // and 48, 16128 53 and 51; 32000 100 and 95)
            if ((int64_t)d.B * d.chunks <= 15 << 10) launch_kernel(k_verify_left<T, 1>, dim3(groups(1), (unsigned)d.B), dim3(VWG), 0, st, d);
            else launch_kernel(k_verify_left<T, 4>, dim3(groups(4), (unsigned)d.B), dim3(VWG), 0, st, d);
            launch_kernel(k_verify_draw<T, false>, dim3((unsigned)d.B), dim3(VWG), 0, st, d);
        } else {
            launch_kernel(k_verify_one<T>, dim3((unsigned)a.B), dim3(VWG),
                          (unsigned)(d.chunks * (sizeof(ChunkStat) + sizeof(double))), st, d);
        }
    });
    return hipGetLastError();
}

}  // namespace qgemv
