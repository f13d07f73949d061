// Products with a rank-r factor, on the tensor cores (tcgen05, bf16, fp32 sums):
//
//   out[i][j] = sum_k A(i, k) B[k][j],   B row-major with r <= 1024 columns
//
//   T = x V, E = dy U    A row-major in i (K-major operand)
//                        (up to 16 rows: on the warp-level MMA, m16n8k16, four
//                        warps sharing 64 columns -- the tcgen05 MMA has 128
//                        rows and one issuer, 400 cycles per 64 columns of the
//                        contraction here against 230 of loads)
//   dU = dy^T T          A row-major in k (M-major operand): no transposed copy
//   dV = (x^)^T E        the same, with A in 8 bits: eight warps expand a tile's
//                        codes to bf16 on its way to the MMA (code * 2^E is
//                        exact for E >= -124; below, its lowest bits are
//                        rounded to multiples of bf16's 2^-133); E comes as
//                        two bf16 terms (high and low part), so that dV's
//                        error is its own rounding, at twice the MMAs of a
//                        product that is small beside the M x N x K ones
//
// B is read as it lies (N-major operand, boxes of 64 columns x 64 rows).
// A CTA owns 128 rows x up to 256 columns of one product and a range of the
// contraction; the CTAs of a cluster (1 to 16) share a tile's contraction
// and add their sums over distributed shared memory in rank order, so there
// are no partial results in memory and the result is reproducible.  The tile
// width and the split are chosen by a cost estimate (choose_tiles): a tile of N
// columns stages (128 + N) x 128 bytes per 64 columns of the contraction
// against 2 N tensor-core cycles, so wide tiles are fed best; short products
// are cut instead, to put every SM to work.
//
//   warp 0  TMA producer;  warp 1  MMA issuer;  warps 2-5  epilogue;
//   warps 2-9  expansion of codes, where there are any;  warps 6-9  quantisation
//   beside few rows
#include <algorithm>
#include <atomic>
#include <cstring>

#include <cuda_fp16.h>

#include "wl_common.cuh"
#include "wl_fp8.h"
#include "wl_fp8_device.cuh"
#include "wl_fp8_encode.cuh"

namespace wl {

namespace {

// warps 2-5 run the epilogue (with few rows the products, too); warps 2-9 expand
// codes, warps 6-9 quantise beside the products of few rows
constexpr int threads_of(int mode) { return mode == kLowrankCodes || mode == kLowrankFew ? 320 : 192; }
constexpr int kExpanders = 8;
constexpr uint32_t kATile = 16384;  // 128 x 64 bf16
constexpr uint32_t kBBox = 8192;    // 64 x 64 bf16
constexpr uint32_t kCodeTile = 8192;  // 64 rows x 128 codes
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 16;

// Descriptor of an M- or N-major bf16 tile: boxes of 64 elements (128 swizzled
// bytes) x 64 contraction rows; 8 rows are 1024 bytes, the next 64 elements one box on.
__device__ __forceinline__ uint64_t mn_major_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(kBBox >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// 16-byte chunk c of row r of a swizzled tile of 128-byte rows.
__device__ __forceinline__ uint32_t chunk_addr(uint32_t tile, int r, int c) { return tile + r * 128 + ((c ^ (r & 7)) << 4); }

// acc[n] += A B for 16 rows x 64 contraction columns of A and the 16 columns of
// B from chunk c0 on.
__device__ __forceinline__ void few_rows_block(uint32_t a_tile, uint32_t b_tile, int c0, int lane, float (&acc)[2][4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t a[4], b[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                     : "r"(chunk_addr(a_tile, lane & 15, 2 * s + (lane >> 4)))
                     : "memory");
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(chunk_addr(b_tile, 16 * s + (lane & 15), c0 + (lane >> 4)))
                     : "memory");
#pragma unroll
        for (int n = 0; n < 2; ++n)
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                : "+f"(acc[n][0]), "+f"(acc[n][1]), "+f"(acc[n][2]), "+f"(acc[n][3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[2 * n]), "r"(b[2 * n + 1]));
    }
}

// Two E4M3 codes (low byte first) times a power of two, as a pair of bf16.
__device__ __forceinline__ uint32_t expand_pair(uint32_t codes, float scale) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h));
    return pack_bf16x2(f.x * scale, f.y * scale);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *dst, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(dst) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void write8(const LowrankJob &jb, int i, int j, const float (&v)[8]) {
    if (i >= jb.I || j >= jb.r) return;
    store8(jb.out + (size_t)i * jb.r + j, v);
    if (jb.out_low) {
        float lo[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) lo[k] = v[k] - __bfloat162float(__float2bfloat16_rn(v[k]));
        store8(jb.out_low + (size_t)i * jb.r + j, lo);
    }
}

// Columns [c0, c1) of the rows whose index is `part` modulo `parts`, by 128
// threads: eight lanes share a block.  c0 is a multiple of 128.
__device__ __forceinline__ void quantize_range(const LowrankQuant &q, int c0, int c1, int part, int parts, int tid) {
    const int pitch = WL_FP8_SCALE_PITCH(q.cols), blocks = (c1 - c0 + 127) / 128;
    const int rows = part < q.rows ? (q.rows - part + parts - 1) / parts : 0;
    const int total = rows * blocks, group = tid >> 3;
    for (int t0 = 0; t0 < total; t0 += 32) {  // 16 groups, two blocks each in flight
        float v[2][16];
        int row[2], c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = t0 + k * 16 + group;
            row[k] = t < total ? part + t / blocks * parts : -1;
            c[k] = c0 + t % blocks * 128 + (tid & 7) * 16;
            Raw16<__nv_bfloat16> raw;
            raw.load(q.a + (size_t)max(row[k], 0) * q.cols + c[k], row[k] >= 0 ? q.cols - c[k] : 0, true);
            raw.unpack(v[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            bool infinities;
            const int E = block_exponent(v[k], infinities);
            if (row[k] < 0) continue;
            if (c[k] < q.cols)
                *reinterpret_cast<uint4 *>(q.codes + (size_t)row[k] * q.cols + c[k]) = codes16(v[k], inverse_scale(E), infinities);
            uint8_t *s = q.scales + (size_t)row[k] * pitch + (c[k] >> 7);
            if ((tid & 7) == 0) *s = (uint8_t)(E + 127);
            // bytes behind the last block
            if ((c[k] >> 7) == (q.cols - 1) >> 7)
                for (int b = (tid & 7) + 1; (c[k] >> 7) + b < pitch; b += 8) s[b] = 127;
        }
    }
}

}  // namespace

template <int kMode>
__global__ void __launch_bounds__(threads_of(kMode), 1) lowrank_kernel(const __grid_constant__ LowrankParams p) {
    constexpr bool kCodes = kMode == kLowrankCodes, kFew = kMode == kLowrankFew, kRows = kFew || kMode == kLowrankRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(base + (size_t)p.stages * p.stage_bytes);
    uint64_t *empty = full + kMaxStages;
    uint64_t *ready = empty + kMaxStages;  // codes expanded
    uint64_t *done = ready + kMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const WaitLimits limits{p.status, p.timeout_ns, abort_flag};

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.split;
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0;
    const int unit = blockIdx.x / S;
    int jx = 0;
    while (jx + 1 < p.njobs && unit >= p.job[jx + 1].tile_begin) ++jx;
    const LowrankJob &jb = p.job[jx];
    const int local = unit - jb.tile_begin;
    const int i_tiles = (jb.I + 127) / 128;
    const int i0 = (local % i_tiles) * 128, j0 = (local / i_tiles) * p.BN;
    const int width = min(p.BN, jb.r - j0), n_mma = (width + 15) & ~15, boxes = (width + 63) / 64;
    const bool quant = kRows && p.quant.a != nullptr;
    int per = (jb.kb + S - 1) / S;
    if (quant) per = (per + 1) & ~1;  // whole 128-column blocks
    const int kb0 = min((int)rank * per, jb.kb), kb1 = min(kb0 + per, jb.kb);
    const int terms = kCodes ? 2 : 1;  // B high, B low

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kFew ? 4 : 1);  // the MMAs' commit, or the warps that read
            mbar_init(&ready[i], kExpanders);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    // Dependents start once everything before this kernel is complete.
    pdl_wait_primary();
    pdl_launch_dependents();
    if (kRows && p.quant.a)
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.quant.n_zero; i += gridDim.x * blockDim.x) p.quant.zero[i] = 0;
    uint32_t tmem = 0;
    if (!kFew) {
        if (warp == 1) {
            tmem_alloc(tmem_slot, p.tmem_cols);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tmem = *tmem_slot;
    }

    const uint32_t a_bytes = kRows ? (uint32_t)p.a_bytes : kATile;
    const uint32_t b_off = a_bytes + (kCodes ? kCodeTile : 0);
    bool ok = true;
    if (warp == 0) {
        Ring r(p.stages);
        uint32_t issued = 0;
        const uint32_t bytes = (kCodes ? kCodeTile : a_bytes) + (uint32_t)(terms * boxes) * kBBox;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = warp_wait(&empty[r.slot], r.phase ^ 1u, limits))) break;
            if (elect_one()) {
                uint8_t *st = base + (size_t)r.slot * p.stage_bytes;
                uint64_t *bar = &full[r.slot];
                mbar_arrive_expect_tx(bar, bytes);
                if (kRows) {
                    tma_load_2d(st, &jb.tm_a, kb * 64, i0, bar);
                } else if (kMode == kLowrankCols) {
                    tma_load_2d(st, &jb.tm_a, i0, kb * 64, bar);
                    tma_load_2d(st + kBBox, &jb.tm_a, i0 + 64, kb * 64, bar);
                } else {
                    tma_load_2d(st + kATile, &jb.tm_a, i0 / 4, kb * 64, bar);  // in words
                }
                for (int b = 0; b < boxes; ++b) {
                    tma_load_2d(st + b_off + b * kBBox, &jb.tm_b, j0 + b * 64, kb * 64, bar);
                    if (kCodes) tma_load_2d(st + b_off + (boxes + b) * kBBox, &jb.tm_b2, j0 + b * 64, kb * 64, bar);
                }
            }
            __syncwarp();
            ++issued;
            r.advance();
        }
        if (!ok && lane == 0) {  // let the copies already issued land before the CTA exits
            const uint32_t left = issued < (uint32_t)p.stages ? issued : p.stages;
            for (uint32_t i = issued - left; i < issued; ++i)
                mbar_wait(&full[i % p.stages], (i / p.stages) & 1u, p.status, 1000000ull);
        }
        __syncwarp();
    } else if (warp == 1 && !kFew) {
        // fp32 sums of bf16 products; A M-major (bit 15) unless its rows run along i; B N-major (bit 16)
        const uint32_t idesc = idesc_bf16_f32(128, n_mma) | (kMode == kLowrankRows ? 0u : 1u << 15) | 1u << 16;
        const uint32_t s0 = smem_addr(base);
        const uint64_t da0 = kMode == kLowrankRows ? sw128_kmajor_desc(s0) : mn_major_desc(s0);
        const uint64_t db0 = mn_major_desc(s0 + b_off), low = ((uint32_t)boxes * kBBox) >> 4;  // B's low term
        const uint64_t step = (uint32_t)p.stage_bytes >> 4;
        constexpr uint64_t kStepA = kMode == kLowrankRows ? 2 : 128;  // 16 contraction rows on: 32 bytes, or 16 rows of 128
        Ring r(p.stages);
        uint32_t acc = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = warp_wait(kCodes ? &ready[r.slot] : &full[r.slot], r.phase, limits))) break;
            tc_fence_after();
            const uint64_t da = da0 + r.slot * step, db = db0 + r.slot * step;
            if (elect_one()) {
                tc_mma_f16(tmem, da, db, idesc, acc);
#pragma unroll
                for (int k = 1; k < 4; ++k) tc_mma_f16(tmem, da + kStepA * k, db + 128 * k, idesc, 1);
                if (kCodes) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_f16(tmem, da + kStepA * k, db + low + 128 * k, idesc, 1);
                }
                tc_commit(&empty[r.slot]);
            }
            __syncwarp();
            acc = 1;
            r.advance();
        }
        if (elect_one()) {
            tc_commit(done);
            // Outstanding MMAs end before TMEM is released, whether or not the
            // epilogue waited for them.
            mbar_wait(done, 0, p.status, kDrainNs);
        }
        __syncwarp();
    } else if (warp > 1) {
        const int tid = threadIdx.x - 64;
        if (kCodes) {
            // 16 codes of one contraction row per step, two steps of 32 rows per
            // block; the next block's scales are on their way meanwhile
            const int k0 = tid >> 3, seg = tid & 7;
            auto scale_of = [&](int kb, int s) -> uint32_t {
                const int m = kb * 64 + s * 32 + k0;
                return m < jb.K ? __ldg(jb.a_scales + (size_t)m * jb.a_pitch + (i0 >> 7)) : 127u;
            };
            uint32_t e[2] = {127u, 127u};
            if (kb0 < kb1) e[0] = scale_of(kb0, 0), e[1] = scale_of(kb0, 1);
            uint32_t slot = 0, ph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                uint32_t next[2] = {127u, 127u};
                if (kb + 1 < kb1) next[0] = scale_of(kb + 1, 0), next[1] = scale_of(kb + 1, 1);
                if (!warp_wait(&full[slot], ph, limits)) {
                    ok = false;
                    break;
                }
                uint8_t *st = base + (size_t)slot * p.stage_bytes;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = s * 32 + k0;
                    const uint4 c = *reinterpret_cast<const uint4 *>(st + kATile + k * 128 + seg * 16);
                    const float sc = scale_value(e[s]);
                    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                    uint32_t o[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[2 * q] = expand_pair(w[q] & 0xFFFFu, sc);
                        o[2 * q + 1] = expand_pair(w[q] >> 16, sc);
                    }
                    // chunk c of 16 bytes of row k sits at c ^ (k & 7)
                    uint8_t *row = st + (seg >> 2) * kBBox + k * 128;
                    const int ch = (seg & 3) * 2;
                    *reinterpret_cast<uint4 *>(row + ((ch ^ (k & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(row + (((ch + 1) ^ (k & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&ready[slot]);
                e[0] = next[0];
                e[1] = next[1];
                if (++slot == (uint32_t)p.stages) slot = 0, ph ^= 1u;
            }
        }
        float few[2][4] = {};  // kFew: columns 16 (warp - 2) .. + 15 of 16 rows
        if (kFew && warp < 6) {
            Ring r(p.stages);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!(ok = warp_wait(&full[r.slot], r.phase, limits))) break;
                const uint32_t st = smem_addr(base) + r.slot * p.stage_bytes;
                few_rows_block(st, st + b_off, 2 * (warp - 2), lane, few);
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[r.slot]);
                r.advance();
            }
        }
        // beside the products of few rows (after them: 36.9 us, beside them 35.0)
        if (quant && (!kFew || warp >= 6))
            quantize_range(p.quant, kb0 * 64, min(kb1 * 64, p.quant.cols), unit, gridDim.x / S, tid & 127);
        // MMAs done.  A CTA with an empty range of the contraction has no sums.
        if (!kFew && ok && warp < 6 && kb1 > kb0) ok = warp_wait(done, 0, limits);
        tc_fence_after();
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16);
        float *buf = reinterpret_cast<float *>(base);  // [column][row], over the idle stages
        if (kFew && warp < 6) {
            // through the exchange buffer, split or not (the stages are idle once all four warps are here)
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    buf[((warp - 2) * 16 + n * 8 + 2 * (lane & 3) + (i & 1)) * 128 + (lane >> 2) + 8 * (i >> 1)] = few[n][i];
        } else if (!kFew && ok && warp < 6)
            for (int c = 0; c < n_mma; c += 8) {
                float v[8];
                if (kb1 > kb0) {
                    uint32_t u[8];
                    tmem_ld8(taddr + c, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(u[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = 0.f;
                }
                if (S == 1) {
                    if (c < width) write8(jb, i0 + row, j0 + c, v);
                } else if (i0 + row < jb.I) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) buf[(c + k) * 128 + row] = v[k];
                }
            }
    }
    tc_fence_before();
    __syncthreads();
    if (!kFew && warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
    if (S > 1 || kFew) {
        __syncwarp();
        cluster_sync();  // every CTA's sums are in its shared memory
        if (warp >= 2 && warp < 6 && ok) {
            const int tid_epilogue = threadIdx.x - 64;
            // groups of eight columns go round the ranks; with few rows several
            // threads take the columns of one row
            const int rows = min(128, jb.I - i0);
            const float *sums = reinterpret_cast<const float *>(base);
            if (rows > 32) {
                const int row = tid_epilogue;
                for (int c = (int)rank * 8; c < width; c += 8 * S) {
                    float v[8] = {};
                    if (row < rows)
                        for (int s = 0; s < S; ++s)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                v[k] += ld_cluster(sums + (c + k) * 128 + row, s);
                    write8(jb, i0 + row, j0 + c, v);
                }
            } else {
                const int groups = (width / 8 - (int)rank + S - 1) / S;
                for (int t = tid_epilogue; t < rows * groups * 8; t += 128) {
                    const int row = t % rows, c = ((int)rank + t / rows / 8 * S) * 8 + t / rows % 8;
                    const float *at = sums + c * 128 + row;
                    float v = 0.f;
                    for (int s0 = 0; s0 < S; s0 += 4) {
                        float part[4];
#pragma unroll
                        for (int s = 0; s < 4; ++s) part[s] = s0 + s < S ? ld_cluster(at, s0 + s) : 0.f;
#pragma unroll
                        for (int s = 0; s < 4; ++s) v += part[s];
                    }
                    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                    const size_t o = (size_t)(i0 + row) * jb.r + j0 + c;
                    jb.out[o] = hi;
                    if (jb.out_low) jb.out_low[o] = __float2bfloat16_rn(v - __bfloat162float(hi));
                }
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while its sums are read
    }
}

// Tile width and split of the contraction, by an estimate of a call's cycles:
// waves of CTAs, each with its blocks of the contraction at the slowest of the
// MMAs (2 cycles per column), the loads (kFp8LowrankFill) and the
// issuing thread (450 cycles), plus 5000 for the start and the drain and, with
// a split, the exchange of 128 x BN sums (60 cycles per column; measured:
// 128 x 256 tiles cut in four took 63 us where whole ones take 28).
static void choose_tiles(LowrankParams &p, int terms, int num_sms) {
    double best = 0;
    const bool few = p.mode == kLowrankFew;
    for (int bn = few ? 64 : 256; bn >= 64; bn /= 2)
        for (int s = 1; s <= kMaxSplit; s *= 2) {
            long long tiles = 0;
            int kb = 0, widest = 0;
            for (int i = 0; i < p.njobs; ++i) {
                tiles += (long long)((p.job[i].I + 127) / 128) * ((p.job[i].r + bn - 1) / bn);
                kb = std::max(kb, p.job[i].kb);
                widest = std::max(widest, p.job[i].r);
            }
            if (bn > 64 && bn / 2 >= widest) continue;
            const int cols = std::min(bn, (widest + 15) / 16 * 16);
            const double loads = (p.a_bytes + 128.0 * cols * terms) / kFp8LowrankFill;
            const double block = few ? loads : std::max({2.0 * cols * terms, loads, 200.0 + 256.0 * terms});
            const double waves = (double)((tiles * s + num_sms - 1) / num_sms);
            const double cost = waves * (((kb + s - 1) / s) * block + 5000 + (s > 1 ? 1000 + 60.0 * cols : 0));
            if (best == 0 || cost < best) {
                best = cost;
                p.BN = bn;
                p.split = s;
            }
        }
}

void plan_fp8_lowrank(LowrankParams &p, LowrankMode mode, int num_sms) {
    if (p.njobs == 0) return;
    const int terms = mode == kLowrankCodes ? 2 : 1;
    int rows = 0;
    for (int i = 0; i < p.njobs; ++i) rows = std::max(rows, lowrank_a_rows(p.job[i].I));
    p.mode = mode == kLowrankRows && rows <= 16 ? kLowrankFew : mode;
    p.a_bytes = mode == kLowrankRows ? rows * 128 : (int)kATile;
    choose_tiles(p, terms, num_sms);
    int widest = 0, longest = 0;
    p.tiles = 0;
    for (int i = 0; i < p.njobs; ++i) {
        LowrankJob &j = p.job[i];
        j.tile_begin = p.tiles;
        p.tiles += (j.I + 127) / 128 * ((j.r + p.BN - 1) / p.BN);
        widest = std::max(widest, j.r);
        longest = std::max(longest, (j.kb + p.split - 1) / p.split);
    }
    const int cols = p.mode == kLowrankFew ? p.BN : std::min((widest + 15) / 16 * 16, p.BN);
    p.stage_bytes = (int)(p.a_bytes + (mode == kLowrankCodes ? kCodeTile : 0) + terms * ((cols + 63) / 64) * kBBox);
    // Narrow tiles leave room for a second CTA on the SM where stages are large:
    // 5376 -> 2 x 21504 at rank 256 and 100 tokens takes 77.3 us with 100 KB, 83.8
    // with 120; 21504 -> 5376 takes 51.4 us with 100 KB, 52.9 with 60.  The stages of
    // up to 16 tokens (10 KB) fill the 100 KB, and with the tail behind them an SM
    // holds one such CTA; 92 KB, which would admit two, are slower (21504 -> 5376 at
    // one token 31.9 us against 31.5) and 123 KB no faster.
    p.stages = std::min(kMaxStages, (p.BN > 64 ? 200 * 1024 : 100 * 1024) / p.stage_bytes);
    p.stages = std::max(2, std::min(p.stages, longest));
    // the exchange of a split tile (and the results of few rows) reuse the stages
    while ((p.split > 1 || p.mode == kLowrankFew) && p.stages * p.stage_bytes < cols * 512) ++p.stages;
    p.tmem_cols = 32;
    while (p.tmem_cols < cols) p.tmem_cols *= 2;
}

cudaError_t launch_fp8_lowrank(const LowrankParams &p, cudaStream_t stream) {
    if (p.njobs == 0) return cudaSuccess;
    const LowrankMode mode = p.mode;
    // an MMA reads 128 rows of A, so the last stage's tile may end behind the stages
    const size_t smem = 1024 + (size_t)p.stages * p.stage_bytes + std::max<size_t>((3 * kMaxStages + 1) * 8 + 32, kATile);
    if (p.stages > kMaxStages || smem > 227 * 1024 || (p.quant.a && mode != kLowrankRows && mode != kLowrankFew))
        return cudaErrorInvalidValue;
    void (*const kernels[4])(LowrankParams) = {lowrank_kernel<kLowrankRows>, lowrank_kernel<kLowrankCols>,
                                               lowrank_kernel<kLowrankCodes>, lowrank_kernel<kLowrankFew>};
    static std::atomic<bool> done[64][4] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev][mode].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernels[mode], cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernels[mode], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done[dev][mode].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.tiles * p.split));
    cfg.blockDim = dim3(threads_of(mode));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernels[mode], p);
}

}  // namespace wl
