// Quantisation to 8 bits: E4M3 codes with one power-of-two scale per block of
// 1 x 128 (activations) or 128 x 128 (weights) elements.
//
// For a block with largest finite magnitude amax, the scale is 2^E with E the
// smallest integer such that 448 * 2^E >= amax: writing amax = (1 + f) 2^e,
// E = e - 8 when 1 + f <= 1.75 (448 = 1.75 * 2^8) and e - 7 otherwise, so E
// comes from the bits of amax and the quotient a * 2^-E is exact.  One
// rounding (to nearest even, by the hardware's conversion) makes the code.
//
// Both kernels read each element once and write one byte for it; the memory
// traffic bounds them.
#include <algorithm>

#include "wl_common.cuh"
#include "wl_fp8.h"
#include "wl_fp8_encode.cuh"

namespace wl {

namespace {

// One warp: 512 columns of one row, 16 per lane, so eight lanes share a block
// and the warp fills one word of scales.  One row per warp: 4096 x 21504 bf16
// take 46 us (5.8 TB/s), 86 with four rows, whose registers cost more warps
// than their loads in flight give.  With column scales neighbouring warps take
// neighbouring rows of the same columns, so the scales (twice the data's bytes
// per element) come from L1.
template <typename T, bool kColScale, bool kMany>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __grid_constant__ Fp8RowsParams p) {
    // Dependents start once everything before this kernel is complete, so they
    // may read its predecessors' results without waiting for this kernel.
    pdl_wait_primary();
    pdl_launch_dependents();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.n_zero; i += (long long)gridDim.x * 256) p.zero[i] = 0;
    long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    int jx = 0;
    if (kMany)
        while (jx + 1 < p.njobs && w >= p.job[jx + 1].warp_begin) ++jx;
    const Fp8RowsJob &jb = p.job[jx];
    const int words = WL_FP8_SCALE_PITCH(jb.cols) / 4;
    w -= jb.warp_begin;
    if (w >= (long long)p.rows * words) return;
    const int row = kColScale ? (int)(w % p.rows) : (int)(w / words), q = kColScale ? (int)(w / p.rows) : (int)(w % words);
    const int c = q * 512 + lane * 16, left = jb.cols - c;
    const T *a = static_cast<const T *>(jb.a) + (size_t)row * jb.lda + c;
    Raw16<T> raw;
    raw.load(a, left, (reinterpret_cast<uintptr_t>(a) & 15u) == 0);
    float v[16];
    raw.unpack(v);
    if constexpr (kColScale) {
        if (jb.copy && c < jb.ld_codes) {  // aligned rows for the kernels that follow
            uint4 *dst = reinterpret_cast<uint4 *>(jb.copy + (size_t)row * jb.ld_codes + c);
            dst[0] = make_uint4(raw.w[0], raw.w[1], raw.w[2], raw.w[3]);
            dst[1] = make_uint4(raw.w[4], raw.w[5], raw.w[6], raw.w[7]);
        }
        const float *cs = jb.colscale + c;
        Raw16<float> s;
        s.load(cs, left, (reinterpret_cast<uintptr_t>(cs) & 15u) == 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= s.f[i];
    }
    bool infinities;
    const int E = block_exponent(v, infinities);
    const uint32_t e = (uint32_t)(E + 127);
    const uint32_t word = __shfl_sync(0xffffffffu, e, 0) | __shfl_sync(0xffffffffu, e, 8) << 8 |
                          __shfl_sync(0xffffffffu, e, 16) << 16 | __shfl_sync(0xffffffffu, e, 24) << 24;
    if (c < jb.ld_codes)
        *reinterpret_cast<uint4 *>(jb.codes + (size_t)row * jb.ld_codes + c) = codes16(v, inverse_scale(E), infinities);
    if (lane == 0) *reinterpret_cast<uint32_t *>(jb.scales + ((size_t)row * words + q) * 4) = word;
}

__device__ __forceinline__ float block_max(float m, float *warp_max) {
    __syncthreads();  // warp_max may still be read
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, warp_max[i]);
    return m;
}

// One CTA: a 128 x 128 block, 16 elements of four rows per thread, kept as
// they are stored so that more CTAs fit an SM.
template <typename T>
__global__ void __launch_bounds__(256, 3) quantize_tiles_kernel(const T *__restrict__ a, int rows, int cols,
                                                             uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                             int pitch) {
    __shared__ float warp_max[8];
    const int c = blockIdx.x * 128 + (threadIdx.x & 7) * 16;
    // a grid has at most 65535 rows of CTAs
    for (int rb = blockIdx.y; rb < (rows + 127) / 128; rb += gridDim.y) {
        const int r0 = rb * 128 + (threadIdx.x >> 3);
        Raw16<T> raw[4];
        float v[16], m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 32 * i;
            raw[i].load(a + (size_t)(r < rows ? r : 0) * cols + c, r < rows ? cols - c : 0, true);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            raw[i].unpack(v);
            m = fmaxf(m, amax16(v));
        }
        m = block_max(m, warp_max);
        const bool infinities = isinf(m);
        if (infinities) {  // the same for the whole block
            m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                raw[i].unpack(v);
                m = fmaxf(m, finite_amax16(v));
            }
            m = block_max(m, warp_max);
        }
        const int E = scale_exponent(m);
        const float inv = inverse_scale(E);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 32 * i;
            raw[i].unpack(v);
            if (r < rows && c < cols) *reinterpret_cast<uint4 *>(codes + (size_t)r * cols + c) = codes16(v, inv, infinities);
        }
        uint8_t *srow = scales + (size_t)rb * pitch;
        if (threadIdx.x == 0) srow[blockIdx.x] = (uint8_t)(E + 127);
        if (blockIdx.x == gridDim.x - 1) {  // bytes behind the last block
            const int b = gridDim.x + threadIdx.x;
            if (b < pitch) srow[b] = 127;
        }
    }
}

__global__ void __launch_bounds__(256) pad_rows_kernel(const __nv_bfloat16 *__restrict__ a, int cols,
                                                       __nv_bfloat16 *__restrict__ out, long long ld) {
    const size_t row = blockIdx.x;
    for (int c = threadIdx.x; c < ld; c += 256)
        out[row * ld + c] = c < cols ? a[row * cols + c] : __float2bfloat16_rn(0.f);
}

}  // namespace

cudaError_t launch_fp8_pad_rows(const __nv_bfloat16 *a, int rows, int cols, __nv_bfloat16 *out, long long ld,
                                cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    pad_rows_kernel<<<rows, 256, 0, stream>>>(a, cols, out, ld);
    return cudaGetLastError();
}

cudaError_t launch_fp8_quantize_rows(Fp8RowsParams &p, wl_type type, cudaStream_t stream) {
    long long warps = 0;
    for (int i = 0; i < p.njobs; ++i) {
        p.job[i].warp_begin = warps;
        warps += (long long)p.rows * (fp8_pitch(p.job[i].cols) / 4);
    }
    if (warps == 0) return cudaSuccess;
    const long long blocks = (warps + 7) / 8;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // several matrices are only ever gradients with their column scales
    void (*const kernel)(Fp8RowsParams) = type == WL_F32 ? quantize_rows_kernel<float, false, false>
                                          : p.job[0].colscale == nullptr ? quantize_rows_kernel<__nv_bfloat16, false, false>
                                                                         : quantize_rows_kernel<__nv_bfloat16, true, true>;
    if (p.njobs > 1 && p.job[0].colscale == nullptr) return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_fp8_quantize_tiles(const void *a, wl_type type, int rows, int cols, uint8_t *codes, uint8_t *scales,
                                      cudaStream_t stream) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const dim3 grid((cols + 127) / 128, std::min((rows + 127) / 128, 65535));
    if (type == WL_BF16)
        quantize_tiles_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16 *>(a), rows, cols, codes, scales,
                                                        fp8_pitch(cols));
    else
        quantize_tiles_kernel<<<grid, 256, 0, stream>>>(static_cast<const float *>(a), rows, cols, codes, scales,
                                                        fp8_pitch(cols));
    return cudaGetLastError();
}

}  // namespace wl
