// Products of the 8-bit operators, one 64 x 64 output tile per CTA, operands
// dequantised to fp32 into shared memory, fp32 multiply-adds.
#include <cuda_fp8.h>

#include "wl_common.cuh"
#include "wl_fp8.h"

namespace wl {

namespace {

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return (float)v;
}

// Operand views: at(i, k) is element (output index i, contraction index k).
struct Rows8 {  // fp8 matrix, 1 x 128 blocks
    Fp8Mat m;
    __device__ float at(int i, int k) const {
        return ldexpf(e4m3_value(m.codes[(size_t)i * m.ld + k]), (int)m.scales[(size_t)i * m.pitch + k / 128] - 127);
    }
};
template <typename V>
struct Transposed {
    V v;
    __device__ float at(int i, int k) const { return v.at(k, i); }
};
struct Bf16 {
    const __nv_bfloat16 *p;
    long long ld;
    __device__ float at(int i, int k) const { return __bfloat162float(p[(size_t)i * ld + k]); }
};

constexpr int kT = 64, kKs = 16;

// acc[a][b] += sum_k A(m0 + 16a + ty, k) B(n0 + 16b + tx, k)
template <typename A, typename B>
__device__ void tile_product(const A &a, const B &b, int M, int N, int K, int m0, int n0, float (&acc)[4][4]) {
    __shared__ float sa[kKs][kT + 1], sb[kKs][kT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < K; k0 += kKs) {
        __syncthreads();
        for (int t = threadIdx.x; t < kKs * kT; t += 256) {
            const int i = t / kKs, k = t % kKs;
            sa[k][i] = m0 + i < M && k0 + k < K ? a.at(m0 + i, k0 + k) : 0.f;
            sb[k][i] = n0 + i < N && k0 + k < K ? b.at(n0 + i, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKs; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(sa[k][16 * x + ty], sb[k][16 * y + tx], acc[x][y]);
    }
}

// out = scale[n] (A1 B1) + A2 B2 (+ acc_in), to bf16 and / or fp32
template <typename A1, typename B1, typename A2, typename B2>
__global__ void __launch_bounds__(256) product_kernel(A1 a1, B1 b1, int K1, const float *scale, A2 a2, B2 b2, int K2,
                                                      int M, int N, float *acc, bool add, __nv_bfloat16 *out) {
    const int m0 = blockIdx.y * kT, n0 = blockIdx.x * kT;
    float p[4][4] = {}, q[4][4] = {};
    tile_product(a1, b1, M, N, K1, m0, n0, p);
    if (K2 > 0) tile_product(a2, b2, M, N, K2, m0, n0, q);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int x = 0; x < 4; ++x)
        for (int y = 0; y < 4; ++y) {
            const int m = m0 + 16 * x + ty, n = n0 + 16 * y + tx;
            if (m >= M || n >= N) continue;
            float v = fmaf(scale ? scale[n] : 1.f, p[x][y], q[x][y]);
            if (add) v += acc[(size_t)m * N + n];
            if (acc) acc[(size_t)m * N + n] = v;
            if (out) out[(size_t)m * N + n] = __float2bfloat16_rn(v);
        }
}

template <typename A1, typename B1, typename A2, typename B2>
cudaError_t product(A1 a1, B1 b1, int K1, const float *scale, A2 a2, B2 b2, int K2, int M, int N, float *acc, bool add,
                    __nv_bfloat16 *out, cudaStream_t stream) {
    if (M == 0 || N == 0) return cudaSuccess;
    const dim3 grid((N + kT - 1) / kT, (M + kT - 1) / kT);
    if (grid.y > 65535) return cudaErrorInvalidValue;
    product_kernel<<<grid, 256, 0, stream>>>(a1, b1, K1, scale, a2, b2, K2, M, N, acc, add, out);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_lowrank(const __nv_bfloat16 *X, long long ldx, int M, int C, const __nv_bfloat16 *V, int r,
                               __nv_bfloat16 *T, cudaStream_t stream) {
    const Bf16 none{nullptr, 0};
    return product(Bf16{X, ldx}, Transposed<Bf16>{{V, r}}, C, nullptr, none, none, 0, M, r, nullptr, false, T, stream);
}

cudaError_t launch_fp8_tn_bf16(const __nv_bfloat16 *X, const __nv_bfloat16 *B, int M, int C, int r,
                               __nv_bfloat16 *out, cudaStream_t stream) {
    const Bf16 none{nullptr, 0};
    return product(Transposed<Bf16>{{X, C}}, Transposed<Bf16>{{B, r}}, M, nullptr, none, none, 0, C, r, nullptr, false,
                   out, stream);
}

cudaError_t launch_fp8_tn_codes(const Fp8Mat &X, const __nv_bfloat16 *B, int M, int C, int r, __nv_bfloat16 *out,
                                cudaStream_t stream) {
    const Bf16 none{nullptr, 0};
    return product(Transposed<Rows8>{{X}}, Transposed<Bf16>{{B, r}}, M, nullptr, none, none, 0, C, r, nullptr, false,
                   out, stream);
}

}  // namespace wl
