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
// Two launches: the chunks of all rows; then, for each sequence, what is accepted
// (found again by every workgroup: a few loads) and the sums of what a refused
// draft leaves of each chunk, after which the workgroup that comes last draws.
// Sums are taken in the order of their places, so the order of arrival changes
// nothing.  Bound by the logits' bytes: the 64-bit exponential of a value, 18
// instructions, takes about 0.7 of the time that its four bytes do.
#include <algorithm>

#include "qgemv_layer.h"

namespace qgemv {

constexpr int VWG = 256;           // threads of a workgroup
constexpr int VWAVES = VWG / 64;
constexpr int VPL = 16;            // values of a chunk a lane
constexpr int VCH = 64 * VPL;      // values of a chunk
constexpr int kOne = 0;            // chunks of a sequence that one workgroup takes by itself

// A chunk of a row: sum of e against its own largest value, which is first at `at`
// (looked for only where the temperature is 0).
struct ChunkStat {
    double sum;
    float top;
    int at;
};

struct VerifyDev {
    const void* logits;
    const int32_t *q_start, *tokens;
    const float *draft, *u, *temperature;
    int32_t *accepted, *next;
    ChunkStat* stats;     // [B][max_q][chunks]
    double* left;         // [B][chunks]
    int* arrived;         // [B]
    int64_t ldl, ldd;
    int T, V, B, max_q, chunks;
};

// The rows of sequence b, and its temperature.
struct Seq {
    int s0, n;
    bool greedy;
    double inv;      // 1 / temperature
};
__device__ __forceinline__ Seq sequence(const VerifyDev& a, int b) {
    Seq s;
    s.s0 = min(max(a.q_start[b], 0), a.T);
    s.n = min(min(max(a.q_start[b + 1], s.s0), a.T) - s.s0, a.max_q);
    const float t = a.temperature ? a.temperature[b] : 1.f;
    s.greedy = !(t > 0.f);
    s.inv = 1.0 / (double)t;
    return s;
}

// exp(y) for y <= 0 from the Taylor series about 0 of what is left of y beside n
// ln 2, |r| <= 0.347: the first term left out is r^13 / 13! < 2^-52.
__device__ __forceinline__ double exponential(double y) {
    y = fmax(y, -800.0);
    const double n = rint(y * 1.4426950408889634);
    const double r = fma(n, 1.7239444525614835e-13, fma(n, -0.6931471805601177, y));   // (ln 2 as 40 bits and the rest: n times the first is exact)
    double p = 1.0 / 479001600.0;
    constexpr double inv[12] = {1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0,
                                1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 12; i++) p = fma(p, r, inv[i]);
    return ldexp(p, (int)n);
}
// e of a logit against the largest, top (not -inf): a -inf has none whatever the
// temperature, and where top is +inf the largest share the mass.
__device__ __forceinline__ double mass(float x, float top, double inv) {
    const double d = (double)x - (double)top;
    return x == top ? 1.0 : d == -INFINITY ? 0.0 : exponential(d * inv);
}
__device__ __forceinline__ float real(float x) { return x == x ? x : -INFINITY; }
template <typename T>
__device__ __forceinline__ float logit(const T* row, int v) {
    return real((float)row[v]);
}

// Sixteen values of chunk c of a row, `none` past its end; value i of lane l is
// number place<T>(c, i) of the row.  (Rows need no alignment beyond their elements'.)
template <typename T>
__device__ __forceinline__ int place(int c, int i) {
    constexpr int G = 16 / sizeof(T);
    return c * VCH + i / G * (64 * G) + (threadIdx.x & 63) * G + i % G;
}
template <typename T>
__device__ __forceinline__ void chunk_values(const T* row, int V, int c, float none, float (&x)[VPL]) {
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
            for (int j = 0; j < G; j++) x[i + j] = v + j < V ? (float)row[v + j] : none;
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

// One chunk of a row, by a wave.
template <typename T>
__device__ __forceinline__ ChunkStat chunk_stat(const VerifyDev& a, const T* row, int c, const Seq& s) {
    float x[VPL];
    chunk_values(row, a.V, c, -INFINITY, x);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        x[i] = real(x[i]);
        top = fmaxf(top, x[i]);
    }
    top = wave_max(top);
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
    for (int i = 0; i < VPL; i++) sum += mass(x[i], top, s.inv);
    r.sum = wave_sum(sum);
    return r;
}

// What a row's chunks say together: its largest value, first at `best`, and the sum.
struct RowStat {
    double sum;
    float top;
    int best;
};
__device__ __forceinline__ double chunk_mass(const ChunkStat& c, float top, double inv) {
    return c.sum > 0.0 ? c.sum * mass(c.top, top, inv) : 0.0;
}
// (by a wave)
__device__ RowStat row_stat(const ChunkStat* stats, int chunks, const Seq& s) {
    const int lane = threadIdx.x & 63;
    float top = -INFINITY;
    for (int c = lane; c < chunks; c += 64) top = fmaxf(top, stats[c].top);
    top = wave_max(top);
    RowStat r{0.0, top, -1};
    if (top == -INFINITY) return r;
    if (s.greedy) {
        int at = INT32_MAX;
        for (int c = lane; c < chunks; c += 64)
            if (stats[c].top == top) at = min(at, stats[c].at);
        r.best = wave_min(at);
        return r;
    }
    double sum = 0.0;
    for (int c = lane; c < chunks; c += 64) sum += chunk_mass(stats[c], top, s.inv);
    r.sum = wave_sum(sum);
    return r;
}
// p of a logit of a row that has mass, and of one of its values.
__device__ __forceinline__ double prob(float x, const RowStat& r, const Seq& s) { return mass(x, r.top, s.inv) / r.sum; }
template <typename T>
__device__ __forceinline__ bool passes(const VerifyDev& a, int row, const RowStat& r, const Seq& s) {
    const int token = a.tokens[row + 1];
    if (token < 0 || token >= a.V) return false;
    const float q = a.draft ? a.draft[(int64_t)(row + 1) * a.ldd + token] : 1.f;
    const double p = s.greedy ? (token == r.best ? 1.0 : 0.0)
                              : r.sum > 0.0 ? prob(logit((const T*)a.logits + (int64_t)row * a.ldl, token), r, s) : 0.0;
    return (double)a.u[row + 1] * (q > 0.f ? (double)q : 0.0) < p;
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
// The sum over a chunk, by a wave, of a row that has mass.
template <typename T>
__device__ double chunk_weight(const VerifyDev& a, Kind kind, int row, int c, const RowStat& r, const Seq& s) {
    float x[VPL], q[VPL] = {};
    chunk_values((const T*)a.logits + (int64_t)row * a.ldl, a.V, c, -INFINITY, x);
    if (kind == kLeft && a.draft) {
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
    for (int i = 0; i < VPL; i++) sum += weight(a, kind, row, place<T>(c, i), x[i], q[i], r, s);
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
        if (found == INT32_MAX && run + w > aim) {
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
    if (!(r.sum > 0.0)) return -1;
    const auto whole = [&](int c) { return chunk_mass(stats[c], r.top, s.inv) / r.sum; };
    if (refused && !a.draft) {
        const int token = a.tokens[row + 1], its = token >= 0 && token < a.V ? token / VCH : -1;
        if (threadIdx.x < 64 && its >= 0) {
            const double w = chunk_weight<T>(a, kLeft, row, its, r, s);
            if (threadIdx.x == 0) rest = w;
        }
        __syncthreads();
        const int next = drawn<T>(a, kLeft, row, u, r, s, [&](int c) { return c == its ? rest : whole(c); });
        if (next >= 0) return next;
    }
    return drawn<T>(a, kWhole, row, u, r, s, whole);
}

// The chunks of all rows, a wave each.
template <typename T>
__global__ __launch_bounds__(VWG) void k_verify_stats(const VerifyDev a) {
    const int c = blockIdx.x * VWAVES + (threadIdx.x >> 6), i = blockIdx.y, b = blockIdx.z;
    if (blockIdx.x == 0 && i == 0 && threadIdx.x == 0) a.arrived[b] = 0;
    const Seq s = sequence(a, b);
    if (i >= s.n || c >= a.chunks) return;
    const ChunkStat r = chunk_stat(a, (const T*)a.logits + (int64_t)(s.s0 + i) * a.ldl, c, s);
    if ((threadIdx.x & 63) == 0) a.stats[((int64_t)b * a.max_q + i) * a.chunks + c] = r;
}

// What is accepted, and the next token.
template <typename T>
__global__ __launch_bounds__(VWG) void k_verify_pick(const VerifyDev a) {
    __shared__ int stop, last;
    __shared__ RowStat at;
    __shared__ double sums[VWAVES];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, b = blockIdx.y;
    const Seq s = sequence(a, b);
    const ChunkStat* stats = a.stats + (int64_t)b * a.max_q * a.chunks;
    // the first row whose draft is refused, four rows at a time: the last row has none
    if (threadIdx.x == 0) stop = s.n > 0 ? s.n - 1 : 0;
    __syncthreads();
    for (int i0 = 0; i0 < s.n; i0 += VWAVES) {
        const int i = i0 + wave;
        RowStat r{};
        bool ends = false;
        if (i < s.n) {
            r = row_stat(stats + (int64_t)i * a.chunks, a.chunks, s);
            ends = i + 1 == s.n || !passes<T>(a, s.s0 + i, r, s);
        }
        if (ends && lane == 0) atomicMin(&stop, i);
        __syncthreads();
        const int now = stop;
        if (ends && i == now && lane == 0) at = r;
        __syncthreads();
        if (now < i0 + VWAVES) break;
    }
    const int done = stop, row = s.s0 + done;
    const RowStat r = at;
    const bool refused = s.n > 0 && done + 1 < s.n;
    int next = -1;
    if (s.n > 0 && !s.greedy && refused && a.draft && r.sum > 0.0) {
        const int c = blockIdx.x * VWAVES + wave;
        if (c < a.chunks) {
            const double w = chunk_weight<T>(a, kLeft, row, c, r, s);
            if (lane == 0) sums[wave] = w;
        }
        __syncthreads();
        double* left = a.left + (int64_t)b * a.chunks;
        if (threadIdx.x == 0) {
            for (int w = 0; w < VWAVES; w++) {
                const int cc = blockIdx.x * VWAVES + w;
                if (cc < a.chunks) __hip_atomic_store(left + cc, sums[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            last = __hip_atomic_fetch_add(a.arrived + b, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        }
        __syncthreads();
        if (!last) return;
        next = drawn<T>(a, kLeft, row, a.u[s.s0], r, s,
                        [&](int cc) { return __hip_atomic_load(left + cc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); });
        if (next < 0) next = drawn_whole<T>(a, false, row, a.u[s.s0], r, s, stats + (int64_t)done * a.chunks);
    } else {
        if (blockIdx.x != 0) return;
        if (s.n > 0)
            next = s.greedy ? r.best : drawn_whole<T>(a, refused, row, a.u[s.s0], r, s, stats + (int64_t)done * a.chunks);
    }
    if (threadIdx.x == 0) {
        a.accepted[b] = done;
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
            const ChunkStat st = chunk_stat(a, (const T*)a.logits + (int64_t)row * a.ldl, c, s);
            if (lane == 0) stats[c] = st;
        }
        __syncthreads();
        const RowStat r = row_stat(stats, a.chunks, s);
        const bool refused = i + 1 < s.n;
        if (refused && passes<T>(a, row, r, s)) {
            done++;
            continue;
        }
        if (s.greedy) {
            next = r.best;
            break;
        }
        const float u = a.u[s.s0];
        if (refused && a.draft && r.sum > 0.0) {
            for (int c = wave; c < a.chunks; c += VWAVES) {
                const double w = chunk_weight<T>(a, kLeft, row, c, r, s);
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
    // the workspace: how many workgroups of a sequence have come, what drafts leave of
    // each chunk, and the chunks of all rows
    const int64_t count = ((int64_t)d.B * 4 + 15) / 16 * 16, left = ((int64_t)d.B * d.chunks * 8 + 15) / 16 * 16;
    const int64_t rows = (int64_t)d.B * d.max_q;
    const int64_t most = std::min<int64_t>(a.ws_bytes, QGEMV_WS_BYTES);
    const bool fits = rows > 0 && count + left <= most && rows <= (most - count - left) / (d.chunks * (int64_t)sizeof(ChunkStat));
    d.arrived = (int*)a.ws;
    d.left = (double*)((char*)a.ws + count);
    d.stats = (ChunkStat*)((char*)a.ws + count + left);
    with_type(a.logits_type, [&](auto t) {
        using T = decltype(t);
        if (fits && (int64_t)d.chunks * d.max_q > kOne) {
            const unsigned x = (unsigned)((d.chunks + VWAVES - 1) / VWAVES);
            launch_kernel(k_verify_stats<T>, dim3(x, (unsigned)d.max_q, (unsigned)d.B), dim3(VWG), 0, st, d);
            launch_kernel(k_verify_pick<T>, dim3(x, (unsigned)d.B), dim3(VWG), 0, st, d);
        } else {
            launch_kernel(k_verify_one<T>, dim3((unsigned)a.B), dim3(VWG),
                          (unsigned)(d.chunks * (sizeof(ChunkStat) + sizeof(double))), st, d);
        }
    });
    return hipGetLastError();
}

}  // namespace qgemv
