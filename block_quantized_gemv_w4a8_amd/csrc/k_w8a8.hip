// k_w8a8.hip -- row quantisation to int8 with one scale per row, and the
// product of int8 codes with one scale per token and per output channel.
#include "qgemv_layer.h"

namespace qgemv {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int QRWG = 256;

// One workgroup per row: the row's largest value, then its codes.  The scale
// and the quotient are correctly rounded divisions, and rounding is half away
// from zero, as in the block quantiser.
template <typename T>
__global__ __launch_bounds__(QRWG) void k_quantize_rows(const T* __restrict__ x, int64_t K,
                                                        int64_t ldx, int8_t* __restrict__ q,
                                                        int64_t ldq, float* __restrict__ sx) {
    __shared__ float part[QRWG / 64];
    const int64_t m = blockIdx.x;
    x += m * ldx;
    q += m * ldq;
    float top = 0.f;
    for (int64_t k = threadIdx.x; k < K; k += QRWG) top = fmaxf(top, fabsf((float)x[k]));
    for (int w = 32; w; w >>= 1) top = fmaxf(top, __shfl_xor(top, w));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float d = top / 127.f;
    if (threadIdx.x == 0) sx[m] = d;
    const int64_t Kp = (K + 15) / 16 * 16;
    for (int64_t k = threadIdx.x; k < Kp; k += QRWG) {
        float c = 0.f;
        if (k < K && d > 0.f) c = fminf(fmaxf(roundf((float)x[k] / d), -127.f), 127.f);
        q[k] = (int8_t)c;
    }
}

hipError_t launch_quantize_rows(const RowsArgs& a, hipStream_t st) {
    with_type(a.x_type, [&](auto t) {
        using T = decltype(t);
        launch_kernel(k_quantize_rows<T>, dim3((unsigned)a.M), dim3(QRWG), 0, st, (const T*)a.x,
                      a.K, a.ldx, a.q, a.ldq, a.sx);
    });
    return hipGetLastError();
}

struct W8Dev {
    const int8_t *w, *q;
    const float *sw, *sx, *bias;
    int64_t ldw, ldq, ldy, N, K, M;
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

// One wave per 16 x 16 tile of y, fragments straight from memory.
template <typename TY>
__global__ __launch_bounds__(64) void k_w8a8(const W8Dev a, TY* __restrict__ y) {
    const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
    const int64_t n0 = 16 * (int64_t)blockIdx.x, m0 = 16 * (int64_t)blockIdx.y;
    const int8_t* w = a.w + min(n0 + r, a.N - 1) * a.ldw;
    const int8_t* q = a.q + min(m0 + r, a.M - 1) * a.ldq;
    i32x4 acc = {0, 0, 0, 0};
    for (int64_t k = 16 * g; k < a.K + 16 * g; k += 64)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(codes16(q, k, a.K), codes16(w, k, a.K), acc, 0,
                                                    0, 0);
    const int64_t n = n0 + r;
    if (n >= a.N) return;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t m = m0 + 4 * g + i;
        if (m >= a.M) continue;
        float f = (float)acc[i] * a.sx[m] * a.sw[n];
        if (a.bias) f += a.bias[n];
        y[m * a.ldy + n] = (TY)f;
    }
}

hipError_t launch_w8a8(const W8A8Args& a, hipStream_t st) {
    const W8Dev d{a.w, a.q, a.sw, a.sx, a.bias, a.ldw, a.ldq, a.ldy, a.N, a.K, a.M};
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 15) / 16));
    with_type(a.y_type, [&](auto t) {
        using TY = decltype(t);
        launch_kernel(k_w8a8<TY>, grid, dim3(64), 0, st, d, (TY*)a.y);
    });
    return hipGetLastError();
}

}  // namespace qgemv
