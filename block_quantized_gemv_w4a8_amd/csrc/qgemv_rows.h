// qgemv_rows.h -- int8 codes of a row with one scale: the arithmetic that row
// quantisation and the 8-bit cache share.
#pragma once

#include "qgemv_layer.h"

namespace qgemv {

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

}  // namespace qgemv
