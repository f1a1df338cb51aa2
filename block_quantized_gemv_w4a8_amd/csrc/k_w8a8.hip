// k_w8a8.hip -- row quantisation to int8 with one scale per row, and the
// product of int8 codes with one scale per token and per output channel.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "qgemv_layer.h"

namespace qgemv {

typedef int i32x4 __attribute__((ext_vector_type(4)));
template <int V> using Int = std::integral_constant<int, V>;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(1))) const void gmem;
typedef __attribute__((address_space(3))) void lmem;

// Row quantisation.  The scale and the quotient are correctly rounded
// divisions, and rounding is half away from zero, as in the block quantiser.
__device__ __forceinline__ float row_scale(float top) { return top / 127.f; }
__device__ __forceinline__ int code(float x, float d) {
    return d > 0.f ? (int)fminf(fmaxf(roundf(x / d), -127.f), 127.f) : 0;
}

// Eight values of a row from 8 c on, those past K zero; p needs no alignment
// beyond its elements'.
template <typename T>
__device__ __forceinline__ void row8(const T* row, int64_t c, int64_t K, float (&f)[8]) {
    T e[8] = {};
    if (8 * c + 8 <= K) {
        __builtin_memcpy(e, row + 8 * c, sizeof e);
    } else if (8 * c < K) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (8 * c + i < K) e[i] = row[8 * c + i];
    }
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = (float)e[i];
}
__device__ __forceinline__ float top8(const float (&f)[8]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(f[i]));
    return top;
}
// Codes of eight values.  A correctly rounded division costs about 25 vector
// instructions a value, more than the row's bytes; but only which side of a
// border h = k + 1/2 the rounded quotient of a = |x| and d falls on is asked.  It
// is h or more where a / d >= h - u / 2, u the spacing of fp32 below h (a tie goes
// to h, whose last bit is 0), so where (a - h d) + d u / 2 >= 0.  h has 8 bits and a
// is near h d where the sign matters, so a - h d is exact in one fma, d u / 2 is a
// power of two times d, and the sum's sign is right.  k = floor(a / d) may be one
// off next to whole numbers, which are far from both borders.  Scales below 2^-100,
// for which d u / 2 would round, and scales that are not finite are divided by.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float d) {
    uint32_t m[8];
    if (d >= 0x1p-100f && d < INFINITY) {
        const float rd = 1.f / d, du = d * 0x1p-24f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float a = fabsf(f[i]), k = floorf(a * rd), h = k + 0.5f;
            const float below = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, h) - 1) & 0x7f800000u);
            const float side = fmaf(du, below, fmaf(-h, d, a));
            const float c = __builtin_copysignf(side >= 0.f ? k + 1.f : k, f[i]);
            m[i] = __builtin_bit_cast(uint32_t, c + 12582912.f);   // (1.5 * 2^23: c is in the low bits)
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) m[i] = (uint32_t)code(f[i], d);
    }
    uint32_t v[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
        v[i] = __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0c0c0400) |
               __builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x04000c0c);
    return make_uint2(v[0], v[1]);
}
template <int W>
__device__ __forceinline__ float row_top(float top, float* part) {
    for (int w = 32; w; w >>= 1) top = fmaxf(top, __shfl_xor(top, w));
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; w++) top = fmaxf(top, part[w]);
    }
    return top;
}

// One workgroup of W waves a row, which holds the row in CH chunks of 8 values
// a thread and reads it once; CH = 0: a row of any length, read twice.  Bound by
// the codes' arithmetic where rows are many (4096 rows of 4096 bf16 values 12.0
// us, 4.2 TB/s; with chunks to spare 14.3, with divisions too 17.7), by the way
// there and back where they are few (one row of 4096 2.4 us, with two passes 8.8).
template <typename T, int W, int CH>
__global__ __launch_bounds__(64 * W) void k_quantize_rows(const T* __restrict__ x, int64_t K,
                                                          int64_t ldx, int8_t* __restrict__ q,
                                                          int64_t ldq, float* __restrict__ sx) {
    __shared__ float part[W];
    const int64_t m = blockIdx.x;
    x += m * ldx;
    uint2* to = reinterpret_cast<uint2*>(q + m * ldq);
    const int64_t chunks = 2 * ((K + 15) / 16);
    float top = 0.f;
    if constexpr (CH > 0) {
        float f[CH][8];
#pragma unroll
        for (int i = 0; i < CH; i++) row8(x, threadIdx.x + 64 * W * i, K, f[i]);
#pragma unroll
        for (int i = 0; i < CH; i++) top = fmaxf(top, top8(f[i]));
        const float d = row_scale(row_top<W>(top, part));
        if (threadIdx.x == 0) sx[m] = d;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const int64_t c = threadIdx.x + 64 * W * i;
            if (c < chunks) to[c] = codes8(f[i], d);
        }
    } else {
        float f[8];
        for (int64_t c = threadIdx.x; c < chunks; c += 64 * W) {
            row8(x, c, K, f);
            top = fmaxf(top, top8(f));
        }
        const float d = row_scale(row_top<W>(top, part));
        if (threadIdx.x == 0) sx[m] = d;
        for (int64_t c = threadIdx.x; c < chunks; c += 64 * W) {
            row8(x, c, K, f);
            to[c] = codes8(f, d);
        }
    }
}

hipError_t launch_quantize_rows(const RowsArgs& a, hipStream_t st) {
    with_type(a.x_type, [&](auto t) {
        using T = decltype(t);
        // (a launch has fewer than 2^32 threads; what is past them would be left out
        // without an error)
        constexpr int64_t kRows = 1 << 21;
        auto go = [&](auto w, auto ch) {
            for (int64_t m = 0; m < a.M; m += kRows)
                launch_kernel(k_quantize_rows<T, w, ch>, dim3((unsigned)std::min(a.M - m, kRows)),
                              dim3(64 * w), 0, st, (const T*)a.x + m * a.ldx, a.K, a.ldx,
                              a.q + m * a.ldq, a.ldq, a.sx + m);
        };
        // few rows: many threads a row; many rows: enough values a thread
        const bool many = a.M > 512;
        if (a.K <= 512) go(Int<1>{}, Int<1>{});
        else if (a.K <= 1024 && many) go(Int<1>{}, Int<2>{});
        else if (a.K <= 2048 && many) go(Int<1>{}, Int<4>{});
        else if (a.K <= 2048) go(Int<4>{}, Int<1>{});
        else if (a.K <= 4096 && many) go(Int<4>{}, Int<2>{});
        else if (a.K <= 8192 && many) go(Int<4>{}, Int<4>{});
        else if (a.K <= 8192) go(Int<16>{}, Int<1>{});
        else if (a.K <= 16384) go(Int<16>{}, Int<2>{});
        else if (a.K <= 32768) go(Int<16>{}, Int<4>{});
        else go(Int<16>{}, Int<0>{});
    });
    return hipGetLastError();
}

struct W8Dev {
    const int8_t *w, *q;
    const float *sw, *sx, *bias;
    int64_t ldw, ldq, ldy, N, K, M;
    int* part;                     // sums split over K: [parts][M][ldp]
    int64_t ldp;
    int tiles_m, tiles_n, group;   // tiles of y, and rows of tiles walked together
    int steps, part_steps;         // steps of 128 codes, and of a part
};

// Sixteen codes of a row, those past K zero.
__device__ __forceinline__ i32x4 codes16(const int8_t* row, int64_t k, int64_t K) {
    i32x4 v = {0, 0, 0, 0};
    if (k < K) v = *reinterpret_cast<const i32x4*>(row + k);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t left = K - k - 4 * i;
        if (left < 4) v[i] = left <= 0 ? 0 : (int)((uint32_t)v[i] & ((1u << (8 * left)) - 1));
    }
    return v;
}

// A tile of y by one workgroup of WM x WN waves: BM tokens, BN channels; the
// workgroup goes on from tile to tile, and the next one's codes are on their way
// while a tile's sums are scaled and stored.
//
// A stage holds 128 codes of every row of the tile: 16-byte chunk c of row r
// sits at place c ^ (r / 2 % 8) of the row, so that the 16 rows of a
// fragment's column of chunks fall on all banks.  Stages go from memory
// straight to LDS, round a ring of RING.  A wave's sums are 32x32x32 tiles with
// the tokens down and the channels across, so that a store has whole runs of
// channels, and a token's runs are stored one after another (with the channels
// down, 16-byte pieces of 32 rows a store, fp32 rows of odd length took 52 us
// where runs take 33: 3539 x 7187 x 306).
//
// Large tiles are bound by the matrix cores at the clock that their power leaves:
// 4096 x 28672 x 4096 takes 470 us, 2050 TOP/s (2110 to 2150 is what the library's
// int8 product reaches, its sums unscaled); the matrix instructions alone, on the
// same codes, run at 2870, and codes of zero at 2450.  Small ones are bound by the way
// from memory to LDS, so they have more stages on their way: 64 x 4096 x 14336
// with a ring of two 35 us, of four 20.
template <int BM, int BN, int WM, int WN, int RING>
struct Tile {
    static constexpr int WAVES = WM * WN;
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int FM = TM / 32, FN = TN / 32;
    static constexpr int STAGE = (BM + BN) * 128;
    static constexpr int LW = BN / 8 / WAVES, LQ = BM / 8 / WAVES;  // 1 KB loads of a stage per wave
    static constexpr int LOADS = LW + LQ;
    static constexpr int SCALES = 2 * BN + (BM < 64 ? 64 : BM);  // sw, bias [BN], sx [BM]
    static constexpr unsigned LDS = RING * STAGE + 2 * 4 * SCALES;
    static_assert(FM * 32 * WM == BM && FN * 32 * WN == BN, "whole fragments");
    static_assert(LW * 8 * WAVES == BN && LQ * 8 * WAVES == BM, "whole loads");
    static constexpr int WGS = 163840 / (int)LDS;        // workgroups that a CU holds
    static_assert(WGS >= 1 && (RING - 1) * LOADS < 60, "a ring that fits, and its loads in flight");
};

// A value of y in fp32.  (It is hidden from the compiler, which would otherwise
// join the last step and the rounding to fp16 in some of the kernels, and the
// same sums would give other bits there.)
__device__ __forceinline__ float y_value(int acc, float sx, float sw, float bias) {
    float f = (float)acc * sx * sw + bias;
    asm("" : "+v"(f));
    return f;
}

// Four channels of a token, of which `left` are there; `to` needs no alignment
// beyond its elements'.
template <typename TY>
__device__ __forceinline__ void put4(TY* to, const float (&f)[4], int64_t left) {
    if (left >= 4) {
        TY e[4];
#pragma unroll
        for (int i = 0; i < 4; i++) e[i] = (TY)f[i];
        __builtin_memcpy(to, e, sizeof e);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (i < left) to[i] = (TY)f[i];
}

// One channel of four tokens, of which `tokens` are there, `left` channels from
// the last; the lane beside has the channel beside (odd: the one before).  Two
// lanes of 16-bit values exchange halves, so that each stores whole pairs.
// WHOLE: all of them are there.
template <bool WHOLE, typename TY>
__device__ __forceinline__ void put_run(TY* to, int64_t ldy, const float (&f)[4], int64_t tokens,
                                        int64_t left, bool odd) {
    if constexpr (sizeof(TY) == 4) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (WHOLE || (i < tokens && left > 0)) to[i * ldy] = f[i];
    } else {
        TY e[4];
#pragma unroll
        for (int i = 0; i < 4; i++) e[i] = (TY)f[i];
        uint32_t a, b;
        __builtin_memcpy(&a, e, 4);
        __builtin_memcpy(&b, e + 2, 4);
        const uint32_t mine = odd ? b : a;
        const uint32_t other = __builtin_amdgcn_mov_dpp(odd ? a : b, 0xb1, 0xf, 0xf, true);  // lane ^ 1
        const uint32_t lo = odd ? other : mine, hi = odd ? mine : other;
        const uint32_t pair[2] = {(lo & 0xffff) | hi << 16, lo >> 16 | (hi & 0xffff0000)};
        to += (odd ? 2 : 0) * ldy - (odd ? 1 : 0);
        tokens -= odd ? 2 : 0;
        left += odd ? 1 : 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (!WHOLE && i >= tokens) continue;
            if (WHOLE || left > 1) __builtin_memcpy(to + i * ldy, &pair[i], 4);
            else if (left == 1) __builtin_memcpy(to + i * ldy, &pair[i], 2);
        }
    }
}

// Orders a block of READS LDS reads, MFMAS matrix instructions and LOADS loads:
// a matrix instruction, which waits for the reads of the block before, then
// reads and loads behind each.
template <int READS, int MFMAS, int LOADS>
__device__ __forceinline__ void interleave() {
    constexpr int per = (READS + MFMAS - 1) / MFMAS, slots = MFMAS - (READS + per - 1) / per;
    constexpr int loads = slots > 0 ? (LOADS + slots - 1) / slots : 0;
#pragma unroll
    for (int i = 0; i < MFMAS; i++) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (i * per < READS) __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
        else if (loads > 0) __builtin_amdgcn_sched_group_barrier(0x20, loads, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Four codes at a time, of which `left` count.
__device__ __forceinline__ int codes_mask(int left) {
    return left >= 4 ? -1 : left <= 0 ? 0 : (int)((1u << (8 * left)) - 1);
}

template <typename TY, int BM, int BN, int WM, int WN, int RING>
__global__ __launch_bounds__(64 * WM * WN, (Tile<BM, BN, WM, WN, RING>::WGS * WM * WN + 3) / 4) void k_w8a8_tile(
    const W8Dev a, TY* __restrict__ y) {
    typedef Tile<BM, BN, WM, WN, RING> S;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r32 = lane & 31, half = lane >> 5;

    const int part = blockIdx.y;
    const int t0 = min(part * a.part_steps, a.steps - 1), n = min(t0 + a.part_steps, a.steps) - t0;
    // codes of this part's last step
    const int last_codes = (int)min(a.K - 128 * (int64_t)(t0 + n - 1), (int64_t)128);
    // (workgroups go round the 8 XCDs: each XCD has a run of tiles of its own,
    // walked in groups of a few rows of tiles)
    const int total = a.tiles_m * a.tiles_n, xcd = blockIdx.x % 8;
    const int tile_end = total / 8 * (xcd + 1) + min(total % 8, xcd + 1);
    const int tile_step = (gridDim.x + 7 - xcd) / 8;
    int tile = total / 8 * xcd + min(total % 8, xcd) + blockIdx.x / 8;
    auto place = [&](int id, int& tm, int& tn) {
        const int group = a.group * a.tiles_n, gi = id / group, first = gi * a.group;
        const int rows = min(a.group, a.tiles_m - first);
        tm = first + (id - gi * group) % rows;
        tn = (id - gi * group) / rows;
    };

    // What is loaded, up to a ring ahead of what is multiplied: this lane's
    // chunk of each load of a stage, as an offset in the tile's rows of one
    // matrix (the launcher holds them below 2^32).
    const int8_t *base_w, *base_q;
    uint32_t off[S::LOADS];
    float* scales = reinterpret_cast<float*>(lds + RING * S::STAGE);   // [2][SCALES]
    int load_tile = tile, load_step = 0, load_side = 0;
    auto row_of = [&](int i) {
        return 8 * (i < S::LW ? S::LW * wave + i : S::LQ * wave + i - S::LW) + (lane >> 3);
    };
    auto chunk_of = [&](int i) { return 16 * ((lane & 7) ^ ((row_of(i) >> 1) & 7)); };
    auto start_tile = [&] {
        int tm, tn;
        place(load_tile, tm, tn);
        const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
        base_w = a.w + n0 * a.ldw + 128 * (int64_t)t0;
        base_q = a.q + m0 * a.ldq + 128 * (int64_t)t0;
        const int last_w = (int)min(a.N - n0, (int64_t)BN) - 1, last_q = (int)min(a.M - m0, (int64_t)BM) - 1;
#pragma unroll
        for (int i = 0; i < S::LOADS; i++)
            off[i] = (i < S::LW ? (uint32_t)min(row_of(i), last_w) * (uint32_t)a.ldw
                                : (uint32_t)min(row_of(i), last_q) * (uint32_t)a.ldq) + chunk_of(i);
        // 64 of the tile's scales a load, by the waves in turn
        for (int i = wave; i < S::SCALES / 64; i += S::WAVES) {
            const int at = 64 * i + lane;
            const bool is_x = 64 * i >= 2 * BN, is_b = !is_x && 64 * i >= BN;
            const float* from =
                is_x ? a.sx + min(m0 + at - 2 * BN, a.M - 1)
                     : (is_b && a.bias ? a.bias : a.sw) + min(n0 + at - (is_b ? BN : 0), a.N - 1);
            __builtin_amdgcn_global_load_lds(
                (gmem*)from, (lmem*)(scales + load_side * S::SCALES + 64 * i), 4, 0, 0);
        }
    };
    // chunks past the row's last one are read from that one (and do not count)
    auto end_row = [&] {
        const int lastc = (last_codes - 1) / 16 * 16;
#pragma unroll
        for (int i = 0; i < S::LOADS; i++) off[i] -= max(chunk_of(i) - lastc, 0);
    };
    auto advance = [&] {
        if (load_step + 1 < n) {
            base_w += 128;
            base_q += 128;
            load_step++;
        } else if (load_tile + tile_step < tile_end) {
            load_tile += tile_step;
            load_side ^= 1;
            load_step = 0;
            start_tile();
        } else {
            return;   // past the last tile: its last stage again, so that a step's loads are always there
        }
        if (load_step == n - 1 && last_codes < 128) end_row();
    };
    auto load = [&](int slot) {
#pragma unroll
        for (int i = 0; i < S::LOADS; i++)
            __builtin_amdgcn_global_load_lds(
                (gmem*)((i < S::LW ? base_w : base_q) + off[i]),
                (lmem*)(lds + slot + (i < S::LW ? 1024 * (S::LW * wave + i)
                                                : 128 * BN + 1024 * (S::LQ * wave + i - S::LW))),
                16, 0, 0);
    };

    i32x16 acc[S::FN][S::FM];
    i32x4 fw[2][S::FN], fq[2][S::FM];
    const int swz = (r32 >> 1) & 7;
    auto read = [&](int slot, int k) {
        const char* st = lds + slot + r32 * 128 + 16 * ((2 * k + half) ^ swz);
#pragma unroll
        for (int n = 0; n < S::FN; n++)
            fw[k & 1][n] = *reinterpret_cast<const i32x4*>(st + (wn * S::TN + 32 * n) * 128);
#pragma unroll
        for (int m = 0; m < S::FM; m++)
            fq[k & 1][m] = *reinterpret_cast<const i32x4*>(st + (BN + wm * S::TM + 32 * m) * 128);
    };
    auto mma = [&](int k) {
#pragma unroll
        for (int n = 0; n < S::FN; n++)
#pragma unroll
            for (int m = 0; m < S::FM; m++)
                acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fq[k & 1][m], fw[k & 1][n],
                                                                  acc[n][m], 0, 0, 0);
    };
    // zeroes the token codes that are past K: nothing else of them counts then
    auto cut = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int mask = codes_mask(last_codes - 32 * k - 16 * half - 4 * i);
#pragma unroll
            for (int m = 0; m < S::FM; m++) fq[k & 1][m][i] &= mask;
        }
    };
    constexpr int READS = S::FN + S::FM, MFMAS = S::FN * S::FM;

    start_tile();
    if (n == 1 && last_codes < 128) end_row();
#pragma unroll
    for (int i = 0; i < RING; i++) {
        if (i) advance();
        load(i * S::STAGE);
    }
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((RING - 1) * S::LOADS) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(0, 0);

    int slot = 0;
    for (int side = 0; tile < tile_end; tile += tile_step, side ^= 1) {
#pragma unroll
        for (int n = 0; n < S::FN; n++)
#pragma unroll
            for (int m = 0; m < S::FM; m++) acc[n][m] = i32x16{};
        // A step of 128 codes: the fragments of 32 are read while those before
        // them are multiplied.  The last 32 are multiplied past the barrier,
        // behind which every wave has read this stage and the next one has
        // landed; the one after that takes this one's place.
        for (int t = 0; t < n; t++) {
            const bool edge = t == n - 1 && last_codes < 128;
#pragma unroll
            for (int k = 0; k < 3; k++) {
                if (edge) cut(k);
                read(slot, k + 1);
                mma(k);
                interleave<READS, MFMAS, 0>();
            }
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((RING - 2) * S::LOADS) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (edge) cut(3);
            advance();
            const int next = slot + S::STAGE < RING * S::STAGE ? slot + S::STAGE : 0;
            read(next, 0);
            load(slot);
            mma(3);
            interleave<READS, MFMAS, S::LOADS>();
            slot = next;
        }
        // (the lane's place is hidden from the compiler here: addresses of this
        // part that are formed before the loop over tiles would not fit the
        // registers beside the sums)
        int r = r32, hh = half;
        asm volatile("" : "+v"(r), "+v"(hh));
        int tm, tn;
        place(tile, tm, tn);
        const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
        const float* sc = scales + side * S::SCALES;
        float sw[S::FN], bias[S::FN];
#pragma unroll
        for (int n = 0; n < S::FN; n++) {
            sw[n] = sc[wn * S::TN + 32 * n + r];
            bias[n] = a.bias ? sc[BN + wn * S::TN + 32 * n + r] : 0.f;
        }
        auto put = [&](auto whole) {
#pragma unroll
            for (int m = 0; m < S::FM; m++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int in = wm * S::TM + 32 * m + 8 * e + 4 * hh;   // of the tile's tokens
                    const f32x4 sx = *reinterpret_cast<const f32x4*>(sc + 2 * BN + in);
#pragma unroll
                    for (int n = 0; n < S::FN; n++) {
                        const int ch = wn * S::TN + 32 * n + r;
                        const i32x4 v = {acc[n][m][4 * e], acc[n][m][4 * e + 1],
                                         acc[n][m][4 * e + 2], acc[n][m][4 * e + 3]};
                        if (a.part) {
                            // (rows of the parts are padded to whole tiles of channels)
                            int* p = a.part + (part * a.M + m0 + in) * a.ldp + n0 + ch;
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                if (whole || m0 + in + i < a.M) p[i * a.ldp] = v[i];
                            continue;
                        }
                        float f[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) f[i] = y_value(v[i], sx[i], sw[n], bias[n]);
                        put_run<whole>(y + (m0 + in) * a.ldy + n0 + ch, a.ldy, f, a.M - m0 - in,
                                       a.N - n0 - ch, r & 1);
                    }
                }
        };
        if (m0 + BM <= a.M && n0 + BN <= a.N) put(std::true_type{});
        else put(std::false_type{});
    }
    // (no load of this workgroup may land in its LDS when that is another's)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Few tokens: a workgroup holds 16 channels and 16 MT tokens, and its waves take
// the runs of 128 codes in turn.  Codes go from memory to registers, in which a
// fragment of the 16x16x64 matrix instruction is 16 codes of one row a lane, U
// runs in flight.  The waves' sums meet in LDS.  Bound by the weights' bytes: 2 x
// 4096 x 14336 takes 13.3 us, 4.4 TB/s (16 x 28672 x 4096, whose token codes are
// as many again from L2, 33.6).
template <typename TY, int MT, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES, MT == 1 ? 8 : 5) void k_w8a8_stream(const W8Dev a,
                                                                           TY* __restrict__ y) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    i32x4* sums = reinterpret_cast<i32x4*>(lds);   // [WAVES][MT][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t m0 = 16 * MT * (int64_t)blockIdx.y, n0 = 16 * (int64_t)blockIdx.x;
    // a row's last chunk stands in for those past it; token codes past K are
    // zeroed, and nothing else counts then
    const int lastc = (int)(a.K - 1) / 16 * 16;
    const int8_t *w = a.w + min(n0 + r, a.N - 1) * a.ldw, *q[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) q[m] = a.q + min(m0 + 16 * m + r, a.M - 1) * a.ldq;
    i32x4 fw[U][2], fq[U][MT][2];
    auto load = [&](int t, int u) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int k = min(128 * t + 64 * i + 16 * g, lastc);
            fw[u][i] = *reinterpret_cast<const i32x4*>(w + k);
#pragma unroll
            for (int m = 0; m < MT; m++) fq[u][m][i] = *reinterpret_cast<const i32x4*>(q[m] + k);
        }
    };
    i32x4 acc[MT] = {};
    auto mma = [&](int t, int u) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (t == a.steps - 1) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int mask = codes_mask((int)a.K - 128 * t - 64 * i - 16 * g - 4 * e);
#pragma unroll
                    for (int m = 0; m < MT; m++) fq[u][m][i][e] &= mask;
                }
            }
#pragma unroll
            for (int m = 0; m < MT; m++)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][i], fq[u][m][i], acc[m], 0, 0, 0);
        }
    };
#pragma unroll
    for (int u = 0; u < U; u++) load(min(wave + u * WAVES, a.steps - 1), u);
    // the scales of the four channels of a token that this thread ends with
    const int vec = threadIdx.x % (64 * MT);
    const int64_t tok = m0 + 16 * (vec / 64) + (vec & 15), c = n0 + 4 * ((vec & 63) >> 4);
    const float sx = a.sx[min(tok, a.M - 1)];
    float sw[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sw[i] = a.sw[min(c + i, a.N - 1)];
        b[i] = a.bias ? a.bias[min(c + i, a.N - 1)] : 0.f;
    }
    for (int t = wave; t < a.steps; t += U * WAVES) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (t + u * WAVES < a.steps) mma(t + u * WAVES, u);
            if (t + (U + u) * WAVES < a.steps) load(t + (U + u) * WAVES, u);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; m++) sums[(wave * MT + m) * 64 + lane] = acc[m];
    __syncthreads();
    if (threadIdx.x >= 64 * MT || tok >= a.M || c >= a.N) return;
    i32x4 sum = sums[vec];
#pragma unroll
    for (int i = 1; i < WAVES; i++) sum += sums[i * 64 * MT + vec];
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = y_value(sum[i], sx, sw[i], b[i]);
    put4(y + tok * a.ldy + c, f, a.N - c);
}

// At most kTokenM rows, from x with their quantisation in the launch or (TX is
// int8_t) from their codes: every workgroup forms the codes in its LDS (the
// first one also writes them out) while its first weight codes are on their
// way.  Otherwise as k_w8a8_stream.  1 x 28672 x 4096 takes 23.0 us from codes,
// 5.1 TB/s, and 24.7 from x in the same run.
constexpr int kTokenM = 2;

template <typename TX, typename TY, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void k_w8a8_token(const W8Dev a, const TX* __restrict__ x,
                                                           int64_t ldx, int8_t* __restrict__ q_out,
                                                           float* __restrict__ sx_out,
                                                           TY* __restrict__ y) {
    constexpr bool kCodes = std::is_same<TX, int8_t>::value;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ float part[kTokenM][WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int M = (int)a.M, row = 128 * a.steps;       // bytes of a row of codes in LDS
    i32x4* sums = reinterpret_cast<i32x4*>(lds + M * row);   // [WAVES][64]
    const int64_t n0 = 16 * (int64_t)blockIdx.x;
    // (x first: loads return in order, and the weights come from further off)
    float f[kTokenM][8];
    if constexpr (!kCodes) {
#pragma unroll
        for (int m = 0; m < kTokenM; m++)
            if (m < M) row8(x + m * ldx, threadIdx.x, a.K, f[m]);
    } else {
        for (int k = threadIdx.x; k < M * (row / 16); k += 64 * WAVES) {
            const int m = k >= row / 16, c = k - m * (row / 16);
            *reinterpret_cast<i32x4*>(lds + 16 * k) = codes16(x + m * ldx, 16 * c, a.K);
        }
    }
    const int lastc = (int)(a.K - 1) / 16 * 16;
    const int8_t* w = a.w + min(n0 + r, a.N - 1) * a.ldw;
    i32x4 fw[U][2];
    auto load = [&](int t, int u) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            fw[u][i] = *reinterpret_cast<const i32x4*>(w + min(128 * t + 64 * i + 16 * g, lastc));
    };
#pragma unroll
    for (int u = 0; u < U; u++) load(min(wave + u * WAVES, a.steps - 1), u);
    // the scales of the four channels of a token that this thread ends with
    const int tok = threadIdx.x & 15;
    const int64_t c = n0 + 4 * ((threadIdx.x & 63) >> 4);
    float sw[4], b[4], sx[kTokenM] = {};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sw[i] = a.sw[min(c + i, a.N - 1)];
        b[i] = a.bias ? a.bias[min(c + i, a.N - 1)] : 0.f;
    }
    if constexpr (kCodes) {
#pragma unroll
        for (int m = 0; m < kTokenM; m++) sx[m] = a.sx[min((int64_t)m, a.M - 1)];
    } else {
        // (a thread's first eight values of a row stay in registers, the others
        // are read again for their codes)
#pragma unroll
        for (int m = 0; m < kTokenM; m++) {
            if (m >= M) continue;
            float top = top8(f[m]);
            for (int64_t k = threadIdx.x + 64 * WAVES; 8 * k < a.K; k += 64 * WAVES) {
                float v[8];
                row8(x + m * ldx, k, a.K, v);
                top = fmaxf(top, top8(v));
            }
            for (int i = 32; i; i >>= 1) top = fmaxf(top, __shfl_xor(top, i));
            if (lane == 0) part[m][wave] = top;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kTokenM; m++) {
            if (m >= M) continue;
            float top = part[m][0];
#pragma unroll
            for (int i = 1; i < WAVES; i++) top = fmaxf(top, part[m][i]);
            sx[m] = row_scale(top);
            const bool out = blockIdx.x == 0;
            if (out && threadIdx.x == 0) sx_out[m] = sx[m];
            for (int k = threadIdx.x; k < row / 8; k += 64 * WAVES) {
                float v[8];
                if (k == (int)threadIdx.x) {
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = f[m][i];
                } else {
                    row8(x + m * ldx, k, a.K, v);
                }
                const uint2 codes = codes8(v, sx[m]);
                *reinterpret_cast<uint2*>(lds + m * row + 8 * k) = codes;
                if (out && 8 * k <= lastc + 8)
                    *reinterpret_cast<uint2*>(q_out + m * a.ldq + 8 * k) = codes;
            }
        }
    }
    __syncthreads();
    const char* q = lds + min(r, M - 1) * row + 16 * g;
    i32x4 acc = {0, 0, 0, 0};
    for (int t = wave; t < a.steps; t += U * WAVES) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int tu = t + u * WAVES;
            if (tu >= a.steps) continue;
#pragma unroll
            for (int i = 0; i < 2; i++)
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    fw[u][i], *reinterpret_cast<const i32x4*>(q + 128 * tu + 64 * i), acc, 0, 0, 0);
            if (tu + U * WAVES < a.steps) load(tu + U * WAVES, u);
        }
    }
    sums[wave * 64 + lane] = acc;
    __syncthreads();
    if (threadIdx.x >= 64 || tok >= M || c >= a.N) return;
    i32x4 sum = sums[lane];
#pragma unroll
    for (int i = 1; i < WAVES; i++) sum += sums[i * 64 + lane];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = y_value(sum[i], tok ? sx[1] : sx[0], sw[i], b[i]);
    put4(y + tok * a.ldy + c, v, a.N - c);
}

// Joins sums that were split over K: four channels of one token a thread, up to
// eight parts in flight (16 parts of 40 x 4096: about 4 us with its launch).
template <typename TY>
__global__ __launch_bounds__(256) void k_w8a8_join(const W8Dev a, int parts, TY* __restrict__ y) {
    const uint32_t runs = (uint32_t)((a.N + 3) / 4), at = blockIdx.x * 256 + threadIdx.x;
    const int64_t tok = at / runs, c = 4 * (int64_t)(at % runs);
    if (tok >= a.M) return;
    const float sx = a.sx[tok];
    float sw[4], b[4], f[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sw[i] = a.sw[min(c + i, a.N - 1)];
        b[i] = a.bias ? a.bias[min(c + i, a.N - 1)] : 0.f;
    }
    i32x4 acc = {0, 0, 0, 0};
    const int* from = a.part + tok * a.ldp + c;
#pragma unroll 8
    for (int p = 0; p < parts; p++) acc += *reinterpret_cast<const i32x4*>(from + p * a.M * a.ldp);
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = y_value(acc[i], sx, sw[i], b[i]);
    put4(y + tok * a.ldy + c, f, a.N - c);
}

constexpr int kCUs = 256;

// How K is split into `want` parts, or fewer: whole steps, as the workspace allows.
static int split(W8Dev& d, int want, const W8A8Args& a, int width) {
    d.ldp = (d.N + width - 1) / width * width;
    const int64_t room = std::min<int64_t>(a.ws_bytes, QGEMV_WS_BYTES) / (4 * d.M * d.ldp);
    int64_t parts = std::max<int64_t>(1, std::min<int64_t>(std::min(want, d.steps), room));
    d.part_steps = (int)((d.steps + parts - 1) / parts);
    parts = (d.steps + d.part_steps - 1) / d.part_steps;
    d.part = parts > 1 ? (int*)a.ws : nullptr;
    return (int)parts;
}

template <typename TY, int BM, int BN, int WM, int WN, int RING>
static void launch_tile(W8Dev d, const W8A8Args& a, int want, TY* y, hipStream_t st) {
    typedef Tile<BM, BN, WM, WN, RING> S;
    d.tiles_m = (int)((d.M + BM - 1) / BM);
    d.tiles_n = (int)((d.N + BN - 1) / BN);
    d.group = std::min(d.tiles_m, 2048 / BM);
    const int parts = split(d, want, a, BN);
    // as many workgroups as the device holds, each with tile after tile; one
    // tile each where it is shorter than the ring
    const int tiles = d.tiles_m * d.tiles_n;
    const int grid = d.part_steps < RING || parts > 1 ? tiles : std::min(tiles, kCUs * S::WGS);
    launch_kernel(k_w8a8_tile<TY, BM, BN, WM, WN, RING>, dim3((unsigned)grid, (unsigned)parts),
                  dim3(64 * S::WAVES), S::LDS, st, d, y);
    if (parts > 1)
        launch_kernel(k_w8a8_join<TY>, dim3((unsigned)((d.M * ((d.N + 3) / 4) + 255) / 256)),
                      dim3(256), 0, st, d, parts, y);
}
template <typename TY, int MT, int WAVES>
static void launch_stream(const W8Dev& d, TY* y, hipStream_t st) {
    launch_kernel(k_w8a8_stream<TY, MT, WAVES, 2>,
                  dim3((unsigned)((d.N + 15) / 16), (unsigned)((d.M + 16 * MT - 1) / (16 * MT))),
                  dim3(64 * WAVES), 1024 * WAVES * MT, st, d, y);
}

// A row or two, while its codes are few beside a workgroup's 16 rows of weights.
// From codes, against k_w8a8_stream: 1 x 28672 x 4096 22.2 us against 26.0, 2 x
// 4096 x 14336 14.7 against 13.3.  With the quantisation in the launch, against
// two launches: 1 x 28672 x 4096 23.6 against 31.0, 2 x 4096 x 4096 7.1 against
// 9.0, 2 x 4096 x 14336 20.5 against 17.9, 4 x 28672 x 4096 37.4 against 33.6.
static bool token_sized(const W8Dev& d) { return d.M <= kTokenM && d.M * d.K <= 16384; }
template <typename TX, typename TY>
static void launch_token(const W8Dev& d, const TX* x, int64_t ldx, int8_t* q, float* sx, TY* y,
                         hipStream_t st) {
    const dim3 grid((unsigned)((d.N + 15) / 16));
    const unsigned codes = (unsigned)(128 * d.steps * d.M);
    // all of a short row is in flight with four waves, and more of them only
    // wait longer for each other (1 x 9728 x 896: 5.8 us, with eight 9.2)
    if (d.K <= 2048)
        launch_kernel(k_w8a8_token<TX, TY, 4, 4>, grid, dim3(256), codes + 4096, st, d, x, ldx, q, sx, y);
    else
        launch_kernel(k_w8a8_token<TX, TY, 8, 4>, grid, dim3(512), codes + 8192, st, d, x, ldx, q, sx, y);
}

// Sixteen waves a workgroup have all of a row of 4096 codes in flight; with few
// codes a wave has too little to do, with many the workgroup's end costs more
// (8 x 14336 x 4096: 16.6 us against 17.4 with eight; 8 x 4096 x 14336: 17.8
// against 16.1).
static bool many_waves(int64_t K) { return K >= 4096 && K <= 8192; }

// Which kernel, and how many parts of K.  The times below are a fit, in
// microseconds, to 120 sizes from 1 x 82 x 170 to 4000 x 14336 x 14336 with
// every tile and split timed: what it chooses takes 2% more than the best on
// average, 20% at most.
struct Choice {
    int tile, parts;
    double us;
};
constexpr int kStreamTile = -1;

static void try_tile(Choice& best, int id, int bm, int bn, int ring, int wgs, const W8Dev& d,
                     int64_t ws_bytes) {
    const double mem = (double)(d.N + d.M) * d.K / 4.2e6;
    const int64_t tiles = (d.M + bm - 1) / bm * ((d.N + bn - 1) / bn);
    const int64_t ldp = (d.N + bn - 1) / bn * bn;
    for (int want = 1; want <= 16; want *= 2) {
        if (want > 1 && (d.steps < 2 * want || 4 * want * d.M * ldp > ws_bytes)) break;
        const int steps = (d.steps + want - 1) / want;
        const double per_cu = std::ceil((double)tiles * want / kCUs);
        const double together = std::min(per_cu, (double)wgs), rounds = per_cu / together;
        // a step takes its matrix instructions and loads, or its share of a
        // load's way through the ring
        const double work = bm * bn * 1.32e-5 + (bm + bn) * 1.46e-3;
        const double step = std::max(together * work, 0.93 / (ring - 1));
        const double cu = rounds * (steps * step + 1.0 + together * bm * bn * 1.33e-4);
        double us = 3.2 + std::sqrt(std::hypot(cu * cu, mem * mem));
        if (want > 1) us += 3.0 + 8.0 * want * d.M * d.N / 6.9e6;
        if (us < best.us) best = Choice{id, want, us};
    }
}
static Choice choose(const W8Dev& d, int64_t ws_bytes) {
    // Up to 16 tokens: a row of tiles would be mostly empty (8 x 4096 x 4096:
    // 7.2 us against 11.1 on tiles; 16 x 28672 x 4096: 33 against 30).  Rows
    // 2^24 bytes apart and more are past the tiles' 32-bit offsets.
    if (d.M <= 16 || std::max(d.ldw, d.ldq) >= (1 << 24)) return Choice{kStreamTile, 1, 0.};
    Choice best{kStreamTile, 1, 1e30};
    if (d.M <= 64) {
        const double groups = std::ceil(d.N / 16.) * std::ceil(d.M / 32.);
        const double full = std::ceil(groups * 8 / (kCUs * 16));
        best.us = 1.4 + groups * d.steps * 128. * (16 + std::min<int64_t>(d.M, 32)) / 11e6 +
                  full * (0.56 * std::ceil(d.steps / 8.) + 1.4);
    }
    ws_bytes = std::min<int64_t>(ws_bytes, QGEMV_WS_BYTES);
    try_tile(best, 0, 256, 256, 2, 1, d, ws_bytes);
    try_tile(best, 1, 256, 128, 3, 1, d, ws_bytes);
    try_tile(best, 2, 128, 128, 4, 1, d, ws_bytes);
    try_tile(best, 3, 128, 64, 3, 2, d, ws_bytes);
    try_tile(best, 4, 64, 64, 4, 2, d, ws_bytes);
    return best;
}

static W8Dev device_args(const W8A8Args& a) {
    W8Dev d{};
    d.w = a.w; d.q = a.q; d.sw = a.sw; d.sx = a.sx; d.bias = a.bias;
    d.ldw = a.ldw; d.ldq = a.ldq; d.ldy = a.ldy; d.N = a.N; d.K = a.K; d.M = a.M;
    d.steps = (int)((d.K + 127) / 128);
    return d;
}

hipError_t launch_w8a8(const W8A8Args& a, hipStream_t st) {
    const W8Dev d = device_args(a);
    const Choice c = choose(d, a.ws_bytes);
    with_type(a.y_type, [&](auto t) {
        using TY = decltype(t);
        TY* y = (TY*)a.y;
        if (c.tile == kStreamTile) {
            if (token_sized(d))
                launch_token<int8_t, TY>(d, d.q, d.ldq, nullptr, nullptr, y, st);
            else if (d.M > 16) launch_stream<TY, 2, 8>(d, y, st);
            else if (many_waves(d.K)) launch_stream<TY, 1, 16>(d, y, st);
            else launch_stream<TY, 1, 8>(d, y, st);
        }
        else if (c.tile == 0) launch_tile<TY, 256, 256, 4, 2, 2>(d, a, c.parts, y, st);
        else if (c.tile == 1) launch_tile<TY, 256, 128, 4, 2, 3>(d, a, c.parts, y, st);
        else if (c.tile == 2) launch_tile<TY, 128, 128, 2, 4, 4>(d, a, c.parts, y, st);
        else if (c.tile == 3) launch_tile<TY, 128, 64, 2, 2, 3>(d, a, c.parts, y, st);
        else launch_tile<TY, 64, 64, 2, 2, 4>(d, a, c.parts, y, st);
    });
    return hipGetLastError();
}

hipError_t launch_quantize_w8a8(const RowsArgs& r, const W8A8Args& a, hipStream_t st) {
    const W8Dev d = device_args(a);
    if (!token_sized(d)) {
        const hipError_t err = launch_quantize_rows(r, st);
        return err != hipSuccess ? err : launch_w8a8(a, st);
    }
    with_type(r.x_type, [&](auto tx) {
        with_type(a.y_type, [&](auto ty) {
            using TX = decltype(tx);
            using TY = decltype(ty);
            launch_token<TX, TY>(d, (const TX*)r.x, r.ldx, r.q, r.sx, (TY*)a.y, st);
        });
    });
    return hipGetLastError();
}

}  // namespace qgemv
