// qgemv_layer.h -- shared by the kernels around the weight products of a
// layer (rotation and cache append, paged attention, int8 token/channel
// products): element types and their conversions, the cache as the kernels
// see it, and the launchers' arguments.  Arguments have passed the gates of
// the public entries.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qgemv_launch.h"

namespace qgemv {

typedef __bf16 bf16;
typedef _Float16 f16;

// Eight consecutive elements as fp32, and back with one rounding (to nearest
// even) each.  p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
    alignas(16) T e[8];
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
        *reinterpret_cast<uint4*>(e + 4) = *reinterpret_cast<const uint4*>(p + 4);
    } else {
        *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = (float)e[i];
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
    alignas(16) T e[8];
#pragma unroll
    for (int i = 0; i < 8; i++) e[i] = (T)f[i];
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<uint4*>(p + 4) = *reinterpret_cast<const uint4*>(e + 4);
}

// Four values in one store, each rounded once (to nearest even).  p is aligned
// to the four.
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&f)[4]) {
    alignas(16) T e[4];
#pragma unroll
    for (int i = 0; i < 4; i++) e[i] = (T)f[i];
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(e);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(e);
}

// Calls f with a value of the element type `type` names.
template <typename F>
inline void with_type(int type, F f) {
    if (type == QGEMV_TYPE_F32) f(float{});
    else if (type == QGEMV_TYPE_F16) f(f16{});
    else f(bf16{});
}
template <typename F>
inline void with_type16(int type, F f) {
    if (type == QGEMV_TYPE_F16) f(f16{});
    else f(bf16{});
}

struct RopeArgs {
    qgemv_kv_cache c;
    int T;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int in_type, q_heads;
    const int32_t* pos;
    const int64_t* slots;
    const float* inv_freq;
    int rot_dim, style;
    void* q_out;
    int64_t ldqo;
};
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st);

struct AttnArgs {
    qgemv_kv_cache c;
    const void* q;
    int T;
    int64_t ldq;
    int q_heads;
    const int32_t* q_start;
    const int32_t* kv_len;
    int B, max_q;
    int64_t max_kv;
    const int32_t* table;
    int64_t ldt;
    float scale;
    int window, sinks;
    void* out;
    int out_type;
    int64_t ldo;
    float* lse;
    void* ws;
    int64_t ws_bytes;
};
hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t st);

struct RowsArgs {
    const void* x;
    int x_type;
    int64_t M, K, ldx;
    int8_t* q;
    int64_t ldq;
    float* sx;
};
hipError_t launch_quantize_rows(const RowsArgs& a, hipStream_t st);

struct W8A8Args {
    const int8_t* w;
    int64_t ldw;
    const float* sw;
    int64_t N, K, M;
    const int8_t* q;
    int64_t ldq;
    const float* sx;
    const float* bias;
    void* y;
    int y_type;
    int64_t ldy;
    void* ws;
    int64_t ws_bytes;
};
hipError_t launch_w8a8(const W8A8Args& a, hipStream_t st);
hipError_t launch_quantize_w8a8(const RowsArgs& r, const W8A8Args& a, hipStream_t st);

}  // namespace qgemv
