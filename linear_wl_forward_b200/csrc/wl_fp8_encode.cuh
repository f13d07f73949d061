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

// 2^(e - 127) of a scale byte: e = 0 is the subnormal 2^-127, 255 the NaN scale.
__device__ __forceinline__ float scale_value(uint32_t e) {
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}

// 2^-E; E in [-127, 120].
__device__ __forceinline__ float inverse_scale(int E) { return __uint_as_float((uint32_t)(127 - E) << 23); }

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : 0.f;  // false for infinities and NaN
}

// Two codes.  NaN gives the NaN code; infinities saturate here (codes16 sees to them).
__device__ __forceinline__ uint32_t code_pair(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

// 16 consecutive elements as they are stored; `n` of them exist, the rest are 0.
// `vec`: p is 16-byte aligned.
template <typename T>
struct Raw16;

template <>
struct Raw16<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int n, bool vec) {
        if (vec && n >= 16) {
            const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = (2 * i < n ? h[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)h[2 * i + 1] << 16 : 0u);
        }
    }
    __device__ __forceinline__ void unpack(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = bf16lo(w[i]);
            v[2 * i + 1] = bf16hi(w[i]);
        }
    }
};

template <>
struct Raw16<float> {
    float f[16];
    __device__ __forceinline__ void load(const float *p, int n, bool vec) {
        if (vec && n >= 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 a = reinterpret_cast<const float4 *>(p)[i];
                f[4 * i] = a.x, f[4 * i + 1] = a.y, f[4 * i + 2] = a.z, f[4 * i + 3] = a.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = i < n ? p[i] : 0.f;
        }
    }
    __device__ __forceinline__ void unpack(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = f[i];
    }
};

// Largest magnitude, NaN left out, infinities not: one instruction per element.
__device__ __forceinline__ float amax16(const float (&v)[16]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));
    return a;
}

// Largest finite magnitude: for blocks that amax16 found an infinity in.
__device__ __forceinline__ float finite_amax16(const float (&v)[16]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, finite_abs(v[i]));
    return a;
}

// `infinities`: some element of the block is infinite; those get the NaN code.
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float inv, bool infinities) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = code_pair(v[4 * i] * inv, v[4 * i + 1] * inv) | code_pair(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    if (infinities) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (isinf(v[i])) w[i >> 2] = (w[i >> 2] & ~(0xFFu << (i & 3) * 8)) | 0x7Fu << (i & 3) * 8;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Maximum over the eight lanes that share a 1 x 128 block.
__device__ __forceinline__ float max_of_8_lanes(float m) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// The scale exponent of a 1 x 128 block held by eight lanes, and whether it
// has infinities.  Called by whole warps.
__device__ __forceinline__ int block_exponent(const float (&v)[16], bool &infinities) {
    float m = max_of_8_lanes(amax16(v));
    infinities = isinf(m);
    if (__any_sync(0xffffffffu, infinities)) m = max_of_8_lanes(finite_amax16(v));
    return scale_exponent(m);
}

}  // namespace wl
