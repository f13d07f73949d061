// Few-token product with 8-bit weights: the weights are the MMA's A operand,
//
//   y[m][n] = s[n] * sum_k 2^(ew + ex) w[n][k] x[m][k]  +  sum_j U[n][j] T[m][j],
//
// so a tile is 128 output rows, its accumulator column a token (Mp = M rounded
// up to 16, at most 128), and a 16 KB block of weights (128 rows x 128
// columns) costs four MMAs of N = Mp.  Reading the weights bounds it: at the
// measured copy rate a block takes each of 148 SMs about 700 cycles.  The
// issuing warp's instructions come next (about 40 cycles per MMA, 70 per wait,
// 46 per commit), so a stage holds two blocks.
//
// A tile is a list of units (the contraction in pairs of blocks, then U's
// 64-column blocks in pairs).  Every CTA, one per SM, takes the same number of
// whole tiles; the tiles left over are cut evenly over the CTAs, so the stream
// has no tail, and done first, so that the exchange hides behind the whole
// ones: a cut tile is summed by the CTA that completes it, from fp32 parts
// s * z + d in CTA order (reproducible).  A call with fewer tiles than SMs gives
// each tile to a cluster (up to 16 CTAs), whose sums meet over distributed
// shared memory, again in rank order.
//
//   warp 0  TMA producer (up to 6 stages of two blocks; without a rank-r launch
//           in front, weights are fetched before the wait for the kernel that makes x)
//   warp 1  MMA issuer;  warp 2  scales;  warps 4-7  epilogue
#include <algorithm>
#include <atomic>

#include "wl_common.cuh"
#include "wl_fp8.h"
#include "wl_fp8_device.cuh"

namespace wl {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kWBytes = 16384;
constexpr uint32_t kSfBytes = 1024;  // four blocks of scales: 128 rows, 128 tokens

__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// A run of units of one tile: [u0, u1) of the tile's own.
struct Segment {
    int seg, tile, u0, u1, nu;  // tile: of its projection; nu: the tile's units
    long long t0;               // first unit of the tile in the call's list
    bool first;                 // the CTA's first piece of the cut tiles
};

__device__ __forceinline__ Segment whole_tile(const Fp8StreamParams &p, int tile) {
    int sp = 0;
    while (sp + 1 < p.nseg && tile >= p.seg[sp + 1].tile_begin) ++sp;
    const Fp8StreamSeg &sg = p.seg[sp];
    const int local = tile - sg.tile_begin;
    return {sp, local, 0, sg.units, sg.units, sg.unit_begin + (long long)local * sg.units, false};
}

// First unit of CTA c's share of the cut tiles.
__device__ __forceinline__ long long cut_begin(const Fp8StreamParams &p, int c) {
    return p.cut_unit + (p.units - p.cut_unit) * min(c, p.cut_ctas) / p.cut_ctas;
}

// The CTA whose share holds unit u of the cut tiles.
__device__ __forceinline__ int cut_cta(const Fp8StreamParams &p, long long u) {
    int c = (int)((u - p.cut_unit) * p.cut_ctas / (p.units - p.cut_unit));
    while (c + 1 < p.cut_ctas && cut_begin(p, c + 1) <= u) ++c;
    while (c > 0 && cut_begin(p, c) > u) --c;
    return c;
}

// The CTA's segments: its share of the cut tiles, then its whole tiles.
struct Walk {
    long long begin, u, end;
    int tile;
    __device__ explicit Walk(const Fp8StreamParams &p)
        : begin(cut_begin(p, blockIdx.x)), u(begin), end(cut_begin(p, blockIdx.x + 1)), tile(blockIdx.x / p.cluster) {}
    __device__ bool next(const Fp8StreamParams &p, Segment &s) {
        if (u < end) {
            int sp = 0;
            while (sp + 1 < p.nseg && u >= p.seg[sp + 1].unit_begin) ++sp;
            const Fp8StreamSeg &sg = p.seg[sp];
            const int tile = (int)((u - sg.unit_begin) / sg.units);
            s = {sp, tile, 0, 0, sg.units, sg.unit_begin + (long long)tile * sg.units, u == begin};
            s.u0 = (int)(u - s.t0);
            s.u1 = (int)min((long long)sg.units, s.u0 + (end - u));
            u += s.u1 - s.u0;
            return true;
        }
        if (tile >= p.whole) return false;
        s = whole_tile(p, tile);
        if (p.cluster > 1) {  // this rank's part of it
            const int rank = (int)cluster_ctarank();
            s.u0 = s.nu * rank / p.cluster;
            s.u1 = s.nu * (rank + 1) / p.cluster;
        }
        tile += gridDim.x / p.cluster;
        return true;
    }
};

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) fp8_stream_kernel(const __grid_constant__ Fp8StreamParams p) {
    if (p.early_next) pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t stages = (uint32_t)p.stages, block_bytes = kWBytes + (uint32_t)p.Mp * 128, stage_bytes = 2 * block_bytes;
    uint8_t *sf_base = base + stages * stage_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(sf_base + 2 * kSfBytes);
    uint64_t *empty = full + stages;
    uint64_t *sf_full = empty + stages;  // [2]
    uint64_t *sf_empty = sf_full + 2;    // [2]
    uint64_t *acc_full = sf_empty + 2;   // [2]
    uint64_t *acc_empty = acc_full + 2;  // [2]
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *last_flag = abort_flag + 1;
    const WaitLimits limits{p.status, p.timeout_ns, abort_flag};

    // TMEM columns: two sums of W0 x, one of U T,
    // two slots of 8 for scales
    const uint32_t set_cols = (uint32_t)max(p.Mp, 32), d_col = 2 * set_cols, sf_col = 3 * set_cols;
    const uint32_t tmem_cols = sf_col + 16 <= 128 ? 128 : sf_col + 16 <= 256 ? 256 : 512;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sf_full[i], 1);
            mbar_init(&sf_empty[i], 1);
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    uint32_t tmem = 0;
    if (warp != 0) {
        pdl_wait_primary();
        if (warp == 1) {
            tmem_alloc(tmem_slot, tmem_cols);
            tmem_relinquish();
        }
        tc_fence_before();
        asm volatile("bar.sync 3, 224;" ::: "memory");  // all but the producer, which is under way
        tc_fence_after();
        tmem = *tmem_slot;
    }

    if (warp == 0) {
        // ------------------------------------------------------ producer ----
        // early: weights of the first `stages` units, then (x made) their operands,
        // then the rest in order; else everything in order once x and T are made
        const uint32_t head = p.early ? stages : 0;
        uint32_t issued = 0;
        bool ok = true;
        for (int pass = p.early ? 0 : 1; pass < 2 && ok; ++pass) {
            // pass 0: weights of units [0, head); pass 1: everything else
            if (pass == 1) pdl_wait_primary();
            uint32_t i = 0, slot = 0, ph = 0;
            Walk walk(p);
            for (Segment s; ok && (pass == 1 || i < head) && walk.next(p, s);) {
                const Fp8StreamSeg &sg = p.seg[s.seg];
                const int n0 = s.tile * 128;
                for (int b = s.u0; b < s.u1 && (pass == 1 || i < head); ++b, ++i) {
                    const bool weights = pass == 0 || i >= head, low = b >= sg.kpairs;
                    // the unit's one or two blocks, `step` columns each
                    const int blk = 2 * (low ? b - sg.kpairs : b), step = low ? 64 : 128;
                    const int two = blk + 1 < (low ? sg.lr : sg.nkb);
                    const CUtensorMap *mw = low ? &p.tm_u[s.seg] : &p.tm_w[s.seg], *mx = low ? &p.tm_t[s.seg] : &p.tm_x;
                    if (i >= head && !warp_wait(&empty[slot], ph ^ 1u, limits)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *st = base + slot * stage_bytes;
                        if (weights) mbar_arrive_expect_tx(&full[slot], block_bytes << two);
                        for (int k = 0; k <= two; ++k) {
                            if (weights) tma_load_2d(st + k * block_bytes, mw, (blk + k) * step, n0, &full[slot]);
                            if (pass == 1) tma_load_2d(st + k * block_bytes + kWBytes, mx, (blk + k) * step, 0, &full[slot]);
                        }
                    }
                    __syncwarp();
                    issued += weights;
                    if (++slot == stages) slot = 0, ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {  // let the copies already issued land before the CTA exits
            const uint32_t left = issued < stages ? issued : stages;
            for (uint32_t i = issued - left; i < issued; ++i)
                mbar_wait(&full[i % stages], (i / stages) & 1u, p.status, 1000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer ---
        const uint32_t idesc0 = idesc_mxf8(128, p.Mp), idesc_lr = idesc_bf16_f32(128, p.Mp);
        const uint64_t da0 = sw128_kmajor_desc(smem_addr(base)), db0 = sw128_kmajor_desc(smem_addr(base) + kWBytes);
        const uint64_t sd0 = scale_desc(smem_addr(sf_base)), next = block_bytes >> 4;
        uint32_t slot = 0, ph = 0, count = 0, chunk = 0;
        bool ok = true;
        Walk walk(p);
        for (Segment s; ok && walk.next(p, s); ++count) {
            const Fp8StreamSeg &sg = p.seg[s.seg];
            const uint32_t set = count & 1u, d_main = tmem + set * set_cols, d_lr = tmem + d_col;
            if (count >= 2) ok = warp_wait(&acc_empty[set], ((count >> 1) - 1) & 1u, limits);
            uint32_t acc = 0;
            for (int b = s.u0; b < s.u1 && ok; ++b) {
                const bool low = b >= sg.kpairs;
                if (low && (b == s.u0 || b == sg.kpairs)) {
                    acc = 0;
                    // the only U T accumulator: read by the segment before
                    if (count >= 1) ok = warp_wait(&acc_empty[set ^ 1u], ((count - 1) >> 1) & 1u, limits);
                }
                const bool scales = !low && (b == s.u0 || (b & 1) == 0);  // of four blocks
                if (scales && ok) {
                    ++chunk;
                    ok = warp_wait(&sf_full[chunk & 1u], ((chunk - 1) >> 1) & 1u, limits);
                }
                if (!ok || !(ok = warp_wait(&full[slot], ph, limits))) break;
                tc_fence_after();
                const uint64_t da = da0 + slot * (stage_bytes >> 4), db = db0 + slot * (stage_bytes >> 4);
                if (low) {
                    const bool two = 2 * (b - sg.kpairs) + 1 < sg.lr;
                    if (elect_one()) {
                        tc_mma_f16(d_lr, da, db, idesc_lr, acc);
#pragma unroll
                        for (int k = 1; k < 4; ++k) tc_mma_f16(d_lr, da + 2 * k, db + 2 * k, idesc_lr, 1);
                        if (two)
#pragma unroll
                            for (int k = 0; k < 4; ++k) tc_mma_f16(d_lr, da + next + 2 * k, db + next + 2 * k, idesc_lr, 1);
                        tc_commit(&empty[slot]);
                    }
                } else {
                    const bool two = 2 * b + 1 < sg.nkb;
                    const uint32_t c = tmem + sf_col + (chunk & 1u) * 8;
                    const uint32_t idesc = idesc0 + (b & 1) * 2 * kScaleByte;  // blocks 2b, 2b + 1 of the chunk's four
                    const uint64_t sd = sd0 + (chunk & 1u) * (kSfBytes >> 4);
                    if (elect_one()) {
                        if (scales) {
                            cp_scales(c, sd);
                            cp_scales(c + 4, sd + (512 >> 4));
                            tc_commit(&sf_empty[chunk & 1u]);
                        }
                        mma_mxf8(d_main, da, db, idesc, c, c + 4, acc);
#pragma unroll
                        for (int k = 1; k < 4; ++k) mma_mxf8(d_main, da + 2 * k, db + 2 * k, idesc, c, c + 4, 1);
                        if (two)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_mxf8(d_main, da + next + 2 * k, db + next + 2 * k, idesc + kScaleByte, c, c + 4, 1);
                        tc_commit(&empty[slot]);
                    }
                }
                __syncwarp();
                acc = 1;
                if (++slot == stages) slot = 0, ph ^= 1u;
            }
            if (ok && elect_one()) tc_commit(&acc_full[set]);
            __syncwarp();
        }
        if (elect_one()) {
            tc_commit(drain);
            mbar_wait(drain, 0, p.status, kDrainNs);  // before TMEM is released
        }
        __syncwarp();
    } else if (warp == 2) {
        // --------------------------------------------------------- scales ---
        uint32_t chunk = 0;
        bool ok = true;
        Walk walk(p);
        for (Segment s; ok && walk.next(p, s);) {
            const Fp8StreamSeg &sg = p.seg[s.seg];
            const uint8_t *wrow = sg.w_scales + (size_t)s.tile * p.pitch;
            for (int b = s.u0; b < min(s.u1, sg.kpairs); b = (b & ~1) + 2) {
                ++chunk;
                const int q = b >> 1;
                const uint32_t ww = __ldg(reinterpret_cast<const uint32_t *>(wrow + 4 * q));
                uint32_t xw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = i * 32 + lane;
                    xw[i] = m < p.M ? __ldg(reinterpret_cast<const uint32_t *>(p.x_scales + (size_t)m * p.pitch + 4 * q)) : 0x7F7F7F7Fu;
                }
                if (chunk > 2) {
                    ok = warp_wait(&sf_empty[chunk & 1u], ((chunk - 3) >> 1) & 1u, limits);
                    if (!ok) break;
                }
                uint8_t *dst = sf_base + (chunk & 1u) * kSfBytes + lane * 16;
                *reinterpret_cast<uint4 *>(dst) = make_uint4(ww, ww, ww, ww);
                *reinterpret_cast<uint4 *>(dst + 512) = make_uint4(xw[0], xw[1], xw[2], xw[3]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sf_full[chunk & 1u]);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------- epilogue ---
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const size_t part_stride = (size_t)p.Mp * 128;
        uint32_t count = 0;
        Walk walk(p);
        for (Segment s; walk.next(p, s); ++count) {
            const Fp8StreamSeg &sg = p.seg[s.seg];
            const uint32_t set = count & 1u;
            // every rank of a cluster leaves its sums for the exchange, also the one
            // that has all units of a short tile beside ranks that have none
            const bool whole = p.cluster == 1 && s.u0 == 0 && s.u1 == s.nu;
            const bool has_z = s.u0 < min(s.u1, sg.kpairs), has_d = s.u1 > max(s.u0, sg.kpairs);  // neither: a rank without units
            bool ok = warp_wait(&acc_full[set], (count >> 1) & 1u, limits);
            {
                // the four warps meet below: they go on, or stop, together
                uint32_t fail;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\t"
                    "setp.ne.u32 p, %1, 0;\n\t"
                    "bar.red.or.pred q, 1, 128, p;\n\t"
                    "selp.u32 %0, 1, 0, q;\n\t}"
                    : "=r"(fail)
                    : "r"((uint32_t)!ok)
                    : "memory");
                if (fail) break;
            }
            tc_fence_after();
            const int n = s.tile * 128 + row;
            const bool in = n < sg.N;
            const float sc = sg.s && in ? __ldg(sg.s + n) : 1.f;
            // which of the CTA's two partial tiles this is: its first, or its last
            // where a piece's sums go: the idle stages, for the cluster, or one of
            // the CTA's two parts in memory
            float *part = p.cluster > 1 ? reinterpret_cast<float *>(base)
                                        : p.parts + ((size_t)blockIdx.x * 2 + (s.first ? 0 : 1)) * part_stride;
            // 16 tokens per step; the stores are predicated, not branched around
            auto drain_tokens = [&](auto store) {
                for (int c = 0; c < p.M; c += 16) {
                    uint32_t z[16], d[16];
                    if (has_z) tmem_ld16(lane_addr + set * set_cols + c, z);
                    if (has_d) tmem_ld16(lane_addr + d_col + c, d);
                    tmem_ld_wait();
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = has_d ? __uint_as_float(d[i]) : 0.f;
                        if (has_z) v[i] = fmaf(sc, __uint_as_float(z[i]), v[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) store(c + i, v[i]);
                }
            };
            if (whole) {
                __nv_bfloat16 *y = sg.y + n;
                const size_t ld = sg.N;
                const int tokens = in ? p.M : 0;
                drain_tokens([&](int m, float v) {
                    if (m < tokens) *y = __float2bfloat16_rn(v);
                    y += ld;
                });
            } else {
                float *q = part + row;
                drain_tokens([&](int m, float v) {
                    if (m < p.M) *q = v;
                    q += 128;
                });
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[set]);
            if (!whole && p.cluster == 1) {
                const int c0 = cut_cta(p, s.t0), c1 = cut_cta(p, s.t0 + s.nu - 1);
                __threadfence();
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (threadIdx.x == 128)
                    *last_flag = atomicAdd(&p.counters[sg.tile_begin + s.tile], 1u) == (unsigned)(c1 - c0);
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (*last_flag) {
                    __threadfence();
                    // the tile is the last piece of its first CTA (or all of
                    // that CTA's share so far), the first piece of the others.
                    // A lane adds four rows of a token, a warp every fourth
                    // token, the parts of four tokens in flight at a time.
                    const float *first = p.parts + ((size_t)c0 * 2 + (cut_begin(p, c0) < s.t0 ? 1 : 0)) * part_stride + lane * 4;
                    const int rows0 = s.tile * 128 + lane * 4;
                    for (int m0 = warp - 4; m0 < p.M; m0 += 16) {
                        float4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = m0 + 4 * i < p.M ? __ldcg(reinterpret_cast<const float4 *>(first + (m0 + 4 * i) * 128)) : make_float4(0, 0, 0, 0);
#pragma unroll 4
                        for (int k = c0 + 1; k <= c1; ++k) {
                            const float *part_k = p.parts + (size_t)k * 2 * part_stride + lane * 4;
                            float4 a[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                a[i] = m0 + 4 * i < p.M ? __ldcg(reinterpret_cast<const float4 *>(part_k + (m0 + 4 * i) * 128)) : make_float4(0, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i].x += a[i].x, v[i].y += a[i].y, v[i].z += a[i].z, v[i].w += a[i].w;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float r[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (m0 + 4 * i < p.M && rows0 + k < sg.N) sg.y[(size_t)(m0 + 4 * i) * sg.N + rows0 + k] = __float2bfloat16_rn(r[k]);
                        }
                    }
                }
                asm volatile("bar.sync 2, 128;" ::: "memory");  // last_flag is used again
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols);
    }
    if (p.cluster > 1) {
        __syncwarp();
        cluster_sync();  // every rank's sums are in its shared memory
        if (warp >= 4) {
            const Segment s = whole_tile(p, blockIdx.x / p.cluster);
            const Fp8StreamSeg &sg = p.seg[s.seg];
            const int row = threadIdx.x - 128, n = s.tile * 128 + row, C = p.cluster;
            const float *sums = reinterpret_cast<const float *>(base) + row;
            // tokens go round the ranks, four at a time
            for (int m0 = (int)cluster_ctarank(); m0 < p.M; m0 += 4 * C) {
                float v[4] = {};
#pragma unroll 4
                for (int r = 0; r < C; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (m0 + i * C < p.M) v[i] += ld_cluster(sums + (m0 + i * C) * 128, r);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (m0 + i * C < p.M && n < sg.N) sg.y[(size_t)(m0 + i * C) * sg.N + n] = __float2bfloat16_rn(v[i]);
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while its sums are read
    }
}

static int fp8_stream_stage(const Fp8StreamParams &p) { return 2 * ((int)kWBytes + p.Mp * 128); }

// More tiles than SMs: whole ones for every CTA, the rest cut.  Fewer: the
// cluster size with the least estimated cycles among those that are resident
// at once, a unit coming at kFp8StreamFill (at 46 bytes per cycle 21504 -> 5376 at
// rank 256 and one token would take clusters of two: 32.9 us against 31.5), or in
// 1400 cycles when all SMs stream, and the exchange taking about 4000 and 30 per
// token.  (5376 x 21504 at one token: 42 tiles whole 37 us, cut over 148 CTAs with
// their parts in memory 31, in clusters of three 22.)
void plan_fp8_stream(Fp8StreamParams &p) {
    constexpr int kSms = kFp8StreamMaxGrid;
    // clusters of 1, 2, .. 16 CTAs, one CTA per SM, that a B200 holds at once
    static const int kResident[kFp8StreamMaxCluster] = {148, 74, 45, 33, 26, 22, 15, 15, 15, 11, 7, 7, 7, 7, 7, 7};
    long long units = 0;
    int tiles = 0, longest = 0;
    for (int i = 0; i < p.nseg; ++i) {
        Fp8StreamSeg &sg = p.seg[i];
        sg.unit_begin = units;
        sg.tile_begin = tiles;
        sg.kpairs = (sg.nkb + 1) / 2;
        sg.units = sg.kpairs + (sg.lr + 1) / 2;
        const int t = (sg.N + 127) / 128;
        tiles += t;
        units += (long long)t * sg.units;
        longest = std::max(longest, sg.units);
    }
    p.units = p.cut_unit = units;
    p.tiles = tiles;
    p.Mp = (p.M + 15) / 16 * 16;
    p.cluster = p.cut_ctas = 1;
    if (tiles <= kSms) {
        p.whole = tiles;
        double least = 0;
        for (int c = 1; c <= kFp8StreamMaxCluster && c <= longest; ++c) {
            if (tiles > kResident[c - 1]) continue;
            const double unit = std::max(fp8_stream_stage(p) / kFp8StreamFill, 1400.0 * c * tiles / kSms);
            const double cost = (longest + c - 1) / c * unit + (c > 1 ? 4000 + 30.0 * p.M : 0);
            if (least == 0 || cost < least) {
                least = cost;
                p.cluster = c;
            }
        }
        p.grid = tiles * p.cluster;
    } else {
        p.whole = tiles / kSms * kSms;
        p.grid = kSms;
        for (int i = 0; i < p.nseg; ++i) {
            const Fp8StreamSeg &sg = p.seg[i];
            const int end = i + 1 < p.nseg ? p.seg[i + 1].tile_begin : tiles;
            if (p.whole >= sg.tile_begin && p.whole < end)
                p.cut_unit = sg.unit_begin + (long long)(p.whole - sg.tile_begin) * sg.units;
        }
        // a share is a good part of a tile, the larger the more tokens a part holds
        const long long share = std::max(2, longest / (p.M <= 16 ? 8 : 4));
        p.cut_ctas = (int)std::min<long long>(kSms, std::max<long long>(1, (units - p.cut_unit) / share));
    }
    // Up to 32 tokens 150 KB hold enough in flight, and more stages gain nothing or
    // lose: 5376 -> 2 x 21504 at one token takes 46.0 us with 150 KB and 49.2 with
    // 200 (39.9 and 42.3 without ranks), 21504 -> 5376 31.5 and 31.3.
    p.stages = std::min(6, ((p.Mp <= 32 ? 150 : 200) * 1024) / fp8_stream_stage(p));
}

size_t fp8_stream_part_floats(const Fp8StreamParams &p) {
    return p.whole == p.tiles ? 0 : (size_t)p.cut_ctas * 2 * p.Mp * 128;
}

cudaError_t launch_fp8_stream(const Fp8StreamParams &p, cudaStream_t stream) {
    if (p.units == 0) return cudaSuccess;
    const size_t smem = 1024 + (size_t)p.stages * fp8_stream_stage(p) + 2 * kSfBytes + (2 * p.stages + 9) * 8 + 16;
    if (p.M < 1 || p.M > kFp8StreamMaxM || smem > 227 * 1024) return cudaErrorInvalidValue;
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fp8_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_stream_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_stream_kernel, p);
}

}  // namespace wl
