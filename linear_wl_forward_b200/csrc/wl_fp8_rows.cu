// The forward of a short call in one launch: a few tokens against at most
// 64 x 148 output rows, small ranks.
//
// Such a call is bound by latency, not by its bytes (Gemma-3-1B's q/k/v are
// 1.8 MB: 0.3 us of memory time), and a chain of dependent launches costs about
// 4 us per link, so every CTA does all of it: it quantises x (M x K, into shared
// memory, as f16 code values and block scales), forms its projection's T = V^T x
// from all of V, and multiplies up to four blocks of 16 rows of W0.  The
// weights of a block's first columns are on their way meanwhile.
//
//   y[m][n] = s[n] * sum over 64-column chunks of 2^(ew + ex) sum_k w x  +  sum_j U[n][j] T[m][j]
//
// E4M3 values are exact in f16, so the products go to the warp-level MMA
// (m16n8k16, fp32 sums) with the rows as M and up to eight tokens as N; the
// contraction's order inside a chunk is free, so a lane's operand is 16
// consecutive bytes of a row.  A chunk has one scale per row block and token,
// applied to its fp32 sums.  Warps take chunks in turn and meet in shared
// memory in a fixed order.
#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "wl_common.cuh"
#include "wl_fp8.h"
#include "wl_fp8_device.cuh"
#include "wl_fp8_encode.cuh"

namespace wl {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTokens = 8;  // the MMA's N
// Rows of V in flight per thread: 9 cover 1152 x 16 in one go, and the fewer
// passes are worth the registers where T is most of the call (1536 x 1152, rank
// 16, one token: 5.9, 5.7, 5.3 and 5.6 us with 4, 6, 9 and 12; 9000 x 640, rank
// 8, which needs three: 5.0, 5.1, 5.4 and 5.6).
constexpr int kAhead = 9;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two codes of a 32-bit word, low or high half, as a pair of f16.
__device__ __forceinline__ uint32_t f16_pair(uint32_t w, int half) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(half ? w >> 16 : w)));
    return h;
}

// The product of two scales as two factors of about the same size: a sum times
// one of them overflows (or loses bits) only where the result does, while the
// scales themselves may cancel (weights of 2^118 with tokens of 2^-118).
__device__ __forceinline__ float2 scale_halves(uint32_t w, uint32_t x) {
    const uint32_t e = w + x, h = e >> 1;
    // the tokens' scales were made here: only the weights' can be NaN
    return make_float2(scale_value(w == 255 ? 255 : h), scale_value(e - h));
}

}  // namespace

// kM: tokens rounded up to 1, 2, 4 or 8;  kBlocks: 16-row blocks per CTA.
template <int kM, int kBlocks>
__global__ void __launch_bounds__(kThreads) fp8_rows_kernel(const __grid_constant__ Fp8RowsForward p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    extern __shared__ __align__(16) uint8_t smem[];
    const int K = p.K, Kp = (K + 63) & ~63, kb = (K + 127) / 128;
    const int ldh = Kp + 8;                                       // halves; rows 16 bytes off 128, for the lanes' reads
    __half *xh = reinterpret_cast<__half *>(smem);                // [kTokens][ldh]
    __nv_bfloat16 *xb = reinterpret_cast<__nv_bfloat16 *>(xh + kTokens * ldh);  // [kM][Kp]
    uint32_t *sx = reinterpret_cast<uint32_t *>(xb + kM * Kp);    // [kTokens][kb] scale bytes
    float *tp = reinterpret_cast<float *>(sx + kTokens * kb);     // [kWarps][kM][32], then T in [0]
    float *zp = tp + kWarps * kM * 32;                            // [kWarps][16 kBlocks][kTokens]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int sp = 0;
    while (sp + 1 < p.nseg && (int)blockIdx.x >= p.seg[sp + 1].cta_begin) ++sp;
    const Fp8RowsSeg &sg = p.seg[sp];
    const int n0 = ((int)blockIdx.x - sg.cta_begin) * 16 * kBlocks;

    // Weights of a chunk: 16 bytes of rows g and g + 8 of every block, and the
    // scale (a CTA's 16, 32 or 64 rows, from a multiple of that, have one).
    uint4 w[kBlocks][2];
    uint32_t ew = 127;
    const uint8_t *w_scales = sg.w_scales + (size_t)(n0 >> 7) * p.pitch;
    auto load_chunk = [&](int c) {
        const int k = c * 64 + t * 16;
        if (c * 64 < K) ew = __ldg(w_scales + (c >> 1));
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = n0 + b * 16 + h * 8 + g;
                w[b][h] = n < sg.N && k < K ? __ldg(reinterpret_cast<const uint4 *>(sg.codes + (size_t)n * K + k)) : make_uint4(0, 0, 0, 0);
            }
    };
    load_chunk(warp);

    // V for T: a thread takes eight columns of every stride-th row, kAhead rows
    // at a time; the first ones are loaded before x is there
    const int groups = sg.r <= 8 ? 1 : sg.r <= 16 ? 2 : 4, j = (lane & (groups - 1)) * 8, stride = kThreads / groups;
    uint4 v[kAhead];
    auto load_v = [&](int k) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i, k += stride)
            v[i] = j < sg.r && k < K ? __ldg(reinterpret_cast<const uint4 *>(sg.V + (size_t)k * sg.r + j)) : make_uint4(0, 0, 0, 0);
    };
    if (sg.r > 0) load_v(threadIdx.x / groups);

    // x: eight lanes per 1 x 128 block
    const int chunk_cols = kb * 128;
    for (int i = threadIdx.x * 16; i < kTokens * chunk_cols; i += kThreads * 16) {
        const int m = i / chunk_cols, c = i - m * chunk_cols;
        Raw16<__nv_bfloat16> raw;
        raw.load(p.x + (size_t)min(m, p.M - 1) * K + c, m < p.M ? K - c : 0, true);
        float e[16];
        raw.unpack(e);
        bool infinities;
        const int E = block_exponent(e, infinities);
        if (c < Kp) {
            const uint4 q = codes16(e, inverse_scale(E), infinities);
            uint4 *dst = reinterpret_cast<uint4 *>(xh + m * ldh + c);
            dst[0] = make_uint4(f16_pair(q.x, 0), f16_pair(q.x, 1), f16_pair(q.y, 0), f16_pair(q.y, 1));
            dst[1] = make_uint4(f16_pair(q.z, 0), f16_pair(q.z, 1), f16_pair(q.w, 0), f16_pair(q.w, 1));
            if (m < kM) {
                uint4 *xd = reinterpret_cast<uint4 *>(xb + m * Kp + c);
                xd[0] = make_uint4(raw.w[0], raw.w[1], raw.w[2], raw.w[3]);
                xd[1] = make_uint4(raw.w[4], raw.w[5], raw.w[6], raw.w[7]);
            }
        }
        if ((threadIdx.x & 7) == 0) sx[m * kb + (c >> 7)] = (uint32_t)(E + 127);
    }
    __syncthreads();

    if (sg.r > 0) {
        float acc[kM][8] = {};
        for (int k0 = threadIdx.x / groups; k0 < K; k0 += kAhead * stride) {
            if (k0 >= stride) load_v(k0);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int k = k0 + q * stride;
                const uint32_t vw[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    const float x = k < K ? __bfloat162float(xb[m * Kp + k]) : 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[m][2 * i] = fmaf(x, bf16lo(vw[i]), acc[m][2 * i]);
                        acc[m][2 * i + 1] = fmaf(x, bf16hi(vw[i]), acc[m][2 * i + 1]);
                    }
                }
            }
        }
        // over the lanes that share the columns (every groups-th)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o >= groups) {
#pragma unroll
                for (int m = 0; m < kM; ++m)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], o);
            }
        if (lane < groups)
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < 8; ++i) tp[(warp * kM + m) * 32 + j + i] = acc[m][i];
    }

    // W0 x
    float z[kBlocks][4] = {};
    const int chunks = Kp / 64;
    for (int c = warp; c < chunks; c += kWarps) {
        uint4 wc[kBlocks][2];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) wc[b][0] = w[b][0], wc[b][1] = w[b][1];
        const uint32_t e = ew;
        if (c + kWarps < chunks) load_chunk(c + kWarps);
        const uint4 *bx = reinterpret_cast<const uint4 *>(xh + g * ldh + c * 64 + t * 16);
        const uint4 b0 = bx[0], b1 = bx[1];
        const uint32_t xb8[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        const float2 f0 = scale_halves(e, sx[2 * t * kb + (c >> 1)]), f1 = scale_halves(e, sx[(2 * t + 1) * kb + (c >> 1)]);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const uint32_t lo[4] = {wc[b][0].x, wc[b][0].y, wc[b][0].z, wc[b][0].w};
            const uint32_t hi[4] = {wc[b][1].x, wc[b][1].y, wc[b][1].z, wc[b][1].w};
            float d[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_f16(d, f16_pair(lo[i], 0), f16_pair(hi[i], 0), f16_pair(lo[i], 1), f16_pair(hi[i], 1), xb8[2 * i], xb8[2 * i + 1]);
            z[b][0] = fmaf(d[0] * f0.x, f0.y, z[b][0]);
            z[b][1] = fmaf(d[1] * f1.x, f1.y, z[b][1]);
            z[b][2] = fmaf(d[2] * f0.x, f0.y, z[b][2]);
            z[b][3] = fmaf(d[3] * f1.x, f1.y, z[b][3]);
        }
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            zp[(warp * 16 * kBlocks + b * 16 + (i >> 1) * 8 + g) * kTokens + 2 * t + (i & 1)] = z[b][i];
    __syncthreads();
    if (sg.r > 0) {
        // T, rounded to bf16 as the tensor-core kernels take it, so that a call with
        // a checkpoint and the same one without differ by the order of sums alone
        for (int i = threadIdx.x; i < kM * 32; i += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) v += tp[q * kM * 32 + i];
            tp[i] = __bfloat162float(__float2bfloat16_rn(v));
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 16 * kBlocks * p.M; i += kThreads) {
        const int row = i % (16 * kBlocks), m = i / (16 * kBlocks), n = n0 + row;
        if (n >= sg.N) continue;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) v += zp[(q * 16 * kBlocks + row) * kTokens + m];
        float d = 0.f;
        for (int j = 0; j < sg.r; j += 8) {
            const uint4 u4 = __ldg(reinterpret_cast<const uint4 *>(sg.U + (size_t)n * sg.r + j));
            const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                d = fmaf(bf16lo(u[k]), tp[m * 32 + j + 2 * k], d);
                d = fmaf(bf16hi(u[k]), tp[m * 32 + j + 2 * k + 1], d);
            }
        }
        sg.y[(size_t)m * sg.N + n] = __float2bfloat16_rn(fmaf(__ldg(sg.s + n), v, d));
    }
}

namespace {
using RowsKernel = void (*)(Fp8RowsForward);
template <int kM>
RowsKernel rows_kernel_of(int blocks) {
    return blocks == 1 ? fp8_rows_kernel<kM, 1> : blocks == 2 ? fp8_rows_kernel<kM, 2> : fp8_rows_kernel<kM, 4>;
}

int tokens_of(int M) { return M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8; }

constexpr size_t rows_smem(int K, int tokens, int blocks) {
    const int Kp = (K + 63) & ~63, kb = (K + 127) / 128;
    return (size_t)kTokens * (Kp + 8) * 2 + (size_t)tokens * Kp * 2 + (size_t)kTokens * kb * 4 + (size_t)kWarps * tokens * 32 * 4 +
           (size_t)kWarps * 16 * blocks * kTokens * 4;
}
constexpr size_t kRowsMaxSmem = rows_smem(kFp8RowsMaxK, kTokens, 4);
static_assert(kRowsMaxSmem <= 227 * 1024, "shared memory of one CTA");
}  // namespace

// Calls that take this kernel: what every CTA repeats (x, V) has to stay small
// beside a launch.  1536 x 1152 with rank 16, against two launches, us: one token
// 5.3 / 9.7, four 6.5 / 9.8, eight 10.9 / 10.0; 2048 x 2048 with rank 32 at one
// token 9.0 / 9.9, at four 11.1 / 10.1; without ranks 4.0 to 7.1 / 8.3.
bool plan_fp8_rows(Fp8RowsForward &p) {
    if (p.M < 1 || p.M > kTokens || p.K > kFp8RowsMaxK) return false;
    int blocks = 0;
    for (int i = 0; i < p.nseg; ++i) {
        const Fp8RowsSeg &sg = p.seg[i];
        if (sg.r > 32 || (long long)tokens_of(p.M) * p.K * sg.r > 96 * 1024) return false;
        blocks += (sg.N + 15) / 16;
    }
    if (blocks > 4 * kFp8StreamMaxGrid) return false;
    p.blocks = blocks <= kFp8StreamMaxGrid ? 1 : blocks <= 2 * kFp8StreamMaxGrid ? 2 : 4;
    p.grid = 0;
    for (int i = 0; i < p.nseg; ++i) {
        p.seg[i].cta_begin = p.grid;
        p.grid += (p.seg[i].N + 16 * p.blocks - 1) / (16 * p.blocks);
    }
    return true;
}

cudaError_t launch_fp8_rows(const Fp8RowsForward &p, cudaStream_t stream) {
    if (p.grid == 0) return cudaSuccess;
    const int tokens = tokens_of(p.M), width = tokens == 1 ? 0 : tokens == 2 ? 1 : tokens == 4 ? 2 : 3;
    const RowsKernel kernel = tokens == 1 ? rows_kernel_of<1>(p.blocks) : tokens == 2 ? rows_kernel_of<2>(p.blocks)
                              : tokens == 4 ? rows_kernel_of<4>(p.blocks) : rows_kernel_of<8>(p.blocks);
    // Raised once per device and kernel, to what any call takes: a limit set for
    // one call would refuse another thread's.
    static std::atomic<bool> done[64][4][3] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::atomic<bool> &raised = done[dev][width][p.blocks >> 1];
    if (!raised.load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsMaxSmem);
        if (e != cudaSuccess) return e;
        raised.store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = rows_smem(p.K, tokens, p.blocks);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace wl
