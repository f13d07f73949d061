// Device-side encoding of blocks in 8 bits: the scale's exponent from a
// block's largest magnitude, and E4M3 codes of elements times 2^-E.
#pragma once

#include "wl_common.cuh"

namespace wl {

// Exponent E of the scale of a block with largest finite magnitude amax >= 0.
__device__ __forceinline__ int scale_exponent(float amax) {
    if (amax == 0.f) return 0;
    const uint32_t b = __float_as_uint(amax);
    if ((b >> 23) == 0) return -127;  // subnormal: E <= -133, clamped
    const int e = (int)(b >> 23) - 127;
    const int E = e - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return E < -127 ? -127 : E;
}

// 2^-E; E in [-127, 120].
__device__ __forceinline__ float inverse_scale(int E) { return __uint_as_float((uint32_t)(127 - E) << 23); }

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : 0.f;  // false for infinities and NaN
}

// Two codes; an element that is not finite becomes the NaN code.
__device__ __forceinline__ uint32_t code_pair(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    uint32_t v = c;
    if (isinf(lo)) v = (v & 0xFF00u) | 0x7Fu;
    if (isinf(hi)) v = (v & 0x00FFu) | 0x7F00u;
    return v;
}

// 16 consecutive elements as floats; `n` of them exist.
template <typename T>
__device__ __forceinline__ void load16(const T *p, int n, bool vec, float (&v)[16]);

template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16 *p, int n, bool vec, float (&v)[16]) {
    if (vec && n >= 16) {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = bf16lo(w[i]);
            v[2 * i + 1] = bf16hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}

template <>
__device__ __forceinline__ void load16<float>(const float *p, int n, bool vec, float (&v)[16]) {
    if (vec && n >= 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 a = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = a.x;
            v[4 * i + 1] = a.y;
            v[4 * i + 2] = a.z;
            v[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}

__device__ __forceinline__ float amax16(const float (&v)[16]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, finite_abs(v[i]));
    return a;
}

__device__ __forceinline__ uint4 codes16(const float (&v)[16], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = code_pair(v[4 * i] * inv, v[4 * i + 1] * inv) | code_pair(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace wl
