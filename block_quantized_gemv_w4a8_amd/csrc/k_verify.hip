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
// A row is taken in chunks of 4096 values, each with its own largest value and sum
// (joined with exp((m - M) / t)), so that sums over chunks give the chunk in which
// the border lies and only that one is walked value by value.
#include <algorithm>

#include "qgemv_layer.h"

namespace qgemv {

constexpr int VWG = 256;           // threads of a workgroup
constexpr int VPT = 16;            // values of a chunk a thread
constexpr int VCH = VWG * VPT;     // values of a chunk

// A chunk of a row: sum of e against its own largest value, which is first at `at`.
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
    ChunkStat* stats;
    double* left;
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

// e of a logit against the largest, top (not -inf): a -inf has none whatever the
// temperature, and where top is +inf the largest share the mass.
__device__ __forceinline__ double mass(float x, float top, double inv) {
    const double d = (double)x - (double)top;
    return x == top ? 1.0 : d == -INFINITY ? 0.0 : exp(d * inv);
}
template <typename T>
__device__ __forceinline__ float logit(const T* row, int v) {
    const float x = (float)row[v];
    return x == x ? x : -INFINITY;
}

template <typename F>
__device__ __forceinline__ double block_sum(double x, double* part, F f) {
    for (int w = 32; w; w >>= 1) x = f(x, __shfl_xor(x, w));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    return f(f(part[0], part[1]), f(part[2], part[3]));
}
__device__ __forceinline__ double block_sum(double x, double* part) {
    return block_sum(x, part, [](double p, double q) { return p + q; });
}

// A value and the place where it stands, larger values and then earlier places first.
__device__ __forceinline__ void larger(float& x, int& at, float y, int there) {
    if (y > x || (y == x && there < at)) {
        x = y;
        at = there;
    }
}

// One chunk of a row, by the workgroup: the same for every thread.
template <typename T>
__device__ ChunkStat chunk_stat(const VerifyDev& a, const T* row, int c, double inv, bool greedy, double* part) {
    float x[VPT];
    const int v0 = c * VCH + 8 * threadIdx.x;     // eight values, and eight more 2048 on
    float top = -INFINITY;
    int at = INT32_MAX;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int v = v0 + i % 8 + i / 8 * (VCH / 2);
        x[i] = v < a.V ? logit(row, v) : -INFINITY;
        if (x[i] > top) {
            top = x[i];
            at = v;
        }
    }
    for (int w = 32; w; w >>= 1) {
        const float y = __shfl_xor(top, w);
        const int there = __shfl_xor(at, w);
        larger(top, at, y, there);
    }
    __shared__ float tops[VWG / 64];
    __shared__ int ats[VWG / 64];
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = top;
        ats[threadIdx.x >> 6] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < VWG / 64; w++) larger(top, at, tops[w], ats[w]);
    ChunkStat s{0.0, top, at};
    if (greedy || top == -INFINITY) return s;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; i++) sum += mass(x[i], top, inv);
    s.sum = block_sum(sum, part);
    return s;
}

// What a row's chunks say together: its largest value, first at `best`, and the sum.
struct RowStat {
    double sum;
    float top;
    int best;
};
__device__ __forceinline__ double chunk_mass(const ChunkStat& s, float top, double inv) {
    return s.top == top ? s.sum : s.sum > 0.0 ? s.sum * mass(s.top, top, inv) : 0.0;
}
__device__ RowStat row_stat(const ChunkStat* stats, int chunks, const Seq& s, double* part) {
    __shared__ float tops[VWG / 64];
    __shared__ int ats[VWG / 64];
    float top = -INFINITY;
    int at = INT32_MAX;
    for (int c = threadIdx.x; c < chunks; c += VWG) larger(top, at, stats[c].top, stats[c].at);
    for (int w = 32; w; w >>= 1) {
        const float y = __shfl_xor(top, w);
        const int there = __shfl_xor(at, w);
        larger(top, at, y, there);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = top;
        ats[threadIdx.x >> 6] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < VWG / 64; w++) larger(top, at, tops[w], ats[w]);
    RowStat r{0.0, top, top == -INFINITY ? -1 : at};
    if (s.greedy || top == -INFINITY) return r;
    double sum = 0.0;
    for (int c = threadIdx.x; c < chunks; c += VWG) sum += chunk_mass(stats[c], top, s.inv);
    r.sum = block_sum(sum, part);
    return r;
}
// p of one value of a row.
template <typename T>
__device__ __forceinline__ double prob(const T* row, int v, const RowStat& r, const Seq& s) {
    if (s.greedy) return v == r.best ? 1.0 : 0.0;
    return r.sum > 0.0 ? mass(logit(row, v), r.top, s.inv) / r.sum : 0.0;
}
__device__ __forceinline__ bool passes(const VerifyDev& a, int row, double p) {
    const float q = a.draft ? a.draft[(int64_t)row * a.ldd + a.tokens[row]] : 1.f;
    return (double)a.u[row] * (q > 0.f ? (double)q : 0.0) < p;
}

// The weights that the next token is drawn by: p, or what the draft leaves of it.
enum Kind { kWhole, kLeft };
template <typename T>
__device__ __forceinline__ double weight(const VerifyDev& a, Kind kind, int row, int v, const RowStat& r, const Seq& s) {
    const double p = prob((const T*)a.logits + (int64_t)row * a.ldl, v, r, s);
    if (kind == kWhole) return p;
    if (!a.draft) return v == a.tokens[row + 1] ? 0.0 : p;
    const float q = a.draft[(int64_t)(row + 1) * a.ldd + v];
    const double w = p - (q > 0.f ? (double)q : 0.0);
    return w > 0.0 ? w : 0.0;
}
template <typename T>
__device__ double chunk_weight(const VerifyDev& a, Kind kind, int row, int c, const RowStat& r, const Seq& s, double* part) {
    double sum = 0.0;
    for (int i = 0; i < VPT; i++) {
        const int v = c * VCH + 8 * (int)threadIdx.x + i % 8 + i / 8 * (VCH / 2);
        if (v < a.V) sum += weight<T>(a, kind, row, v, r, s);
    }
    return block_sum(sum, part);
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
    for (int w = 0; w < VWG / 64; w++) {
        if (w < wave) head += part[w];
        total += part[w];
    }
    return head + sum - x;
}
// The smallest (or largest) of the threads' numbers.
__device__ int least(int x, int* part) {
    for (int w = 32; w; w >>= 1) x = min(x, __shfl_xor(x, w));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    return min(min(part[0], part[1]), min(part[2], part[3]));
}

// The token that is drawn from the weights of a row whose chunks' sums are in `sums`,
// -1 if they are all 0.
template <typename T>
__device__ int drawn(const VerifyDev& a, Kind kind, int row, float u, const RowStat& r, const Seq& s, const double* sums,
                     double* part, int* ipart) {
    const int each = (a.chunks + VWG - 1) / VWG, c0 = threadIdx.x * each, c1 = min(c0 + each, a.chunks);
    double own = 0.0, total;
    for (int c = c0; c < c1; c++) own += sums[c];
    double run = before(own, total, part);
    if (!(total > 0.0)) return -1;
    const double aim = u > 0.f ? (double)u * total : 0.0;
    int found = INT32_MAX, last = INT32_MAX;     // (last: counted from the end)
    double base = 0.0;
    for (int c = c0; c < c1; c++) {
        if (sums[c] > 0.0) last = a.chunks - 1 - c;
        if (found == INT32_MAX && run + sums[c] > aim) {
            found = c;
            base = run;
        }
        run += sums[c];
    }
    const int first = least(found, ipart);
    const int end = a.chunks - 1 - least(last, ipart);
    const bool none = first == INT32_MAX;
    const int c = none ? end : first;
    __shared__ double start;
    if (!none && found == first) start = base;
    __syncthreads();
    const double from = none ? 0.0 : start;
    // value by value: each thread has a run of them
    double w[VPT];
    own = 0.0;
    for (int i = 0; i < VPT; i++) {
        const int v = c * VCH + VPT * (int)threadIdx.x + i;
        w[i] = v < a.V ? weight<T>(a, kind, row, v, r, s) : 0.0;
        own += w[i];
    }
    double chunk;
    run = from + before(own, chunk, part);
    found = last = INT32_MAX;
    for (int i = 0; i < VPT; i++) {
        const int v = VPT * (int)threadIdx.x + i;
        run += w[i];
        if (w[i] > 0.0) last = VCH - 1 - v;
        if (!none && found == INT32_MAX && run > aim && w[i] > 0.0) found = v;
    }
    const int at = least(found, ipart), tail = least(last, ipart);
    return c * VCH + (at != INT32_MAX ? at : tail != INT32_MAX ? VCH - 1 - tail : 0);
}

// A sequence by one workgroup, row by row.
template <typename T>
__global__ __launch_bounds__(VWG) void k_verify_one(const VerifyDev a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    ChunkStat* stats = reinterpret_cast<ChunkStat*>(lds);
    double* sums = reinterpret_cast<double*>(lds + (size_t)a.chunks * sizeof(ChunkStat));
    __shared__ double part[VWG / 64];
    __shared__ int ipart[VWG / 64];
    const int b = blockIdx.x;
    const Seq s = sequence(a, b);
    int done = 0, next = -1;
    for (int i = 0; i < s.n; i++) {
        const int row = s.s0 + i;
        const T* x = (const T*)a.logits + (int64_t)row * a.ldl;
        __syncthreads();
        for (int c = 0; c < a.chunks; c++) {
            const ChunkStat st = chunk_stat(a, x, c, s.inv, s.greedy, part);
            if (threadIdx.x == 0) stats[c] = st;
        }
        __syncthreads();
        const RowStat r = row_stat(stats, a.chunks, s, part);
        if (i + 1 < s.n) {
            const int token = a.tokens[row + 1];
            if (token >= 0 && token < a.V && passes(a, row + 1, prob(x, token, r, s))) {
                done++;
                continue;
            }
        }
        if (s.greedy) {
            next = r.best;
            break;
        }
        const float u = a.u[s.s0];
        if (i + 1 < s.n) {
            for (int c = 0; c < a.chunks; c++) {
                const double w = chunk_weight<T>(a, kLeft, row, c, r, s, part);
                if (threadIdx.x == 0) sums[c] = w;
            }
            __syncthreads();
            next = drawn<T>(a, kLeft, row, u, r, s, sums, part, ipart);
        }
        if (next < 0 && r.sum > 0.0) {
            __syncthreads();
            for (int c = threadIdx.x; c < a.chunks; c += VWG) sums[c] = chunk_mass(stats[c], r.top, s.inv) / r.sum;
            __syncthreads();
            next = drawn<T>(a, kWhole, row, u, r, s, sums, part, ipart);
        }
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
    with_type(a.logits_type, [&](auto t) {
        using T = decltype(t);
        launch_kernel(k_verify_one<T>, dim3((unsigned)a.B), dim3(VWG),
                      (unsigned)(d.chunks * (sizeof(ChunkStat) + sizeof(double))), st, d);
    });
    return hipGetLastError();
}

}  // namespace qgemv
