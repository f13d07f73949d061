// Block-scaled 8-bit GEMM on CTA pairs (tcgen05, cta_group::2):
//
//   out[m][n] = s[n] * sum_k 2^(ea + eb) a[m][k] b[n][k]  +  sum_j T[m][j] U[n][j]
//
// with E4M3 codes a, b and one E8M0 scale per 128 columns of the contraction
// (per row of A, per 128 rows of B).  The scales are powers of two, so the
// block-scaled MMA (kind::mxf8f6f4, which takes one scale per row and 32
// columns) applies them at full rate and the sum over all of the contraction
// stays in TMEM; each 128-column block issues four MMAs that select the same
// scale byte.  The rank-r term is bf16 (kind::f16) into an accumulator of its
// own, since s scales the first sum alone.
//
// A CTA pair owns a 256 x 224 tile: each CTA stages 128 rows of A and 112 of
// B per block (30 KB against 448 tensor-core cycles; a 128 x 256 tile of one
// CTA would stage 48 KB against 512).  An SM takes in about 46 bytes per cycle,
// so the loads (650 cycles per block) bound long products.  224 columns,
// because two accumulators of that width and the scales fit the 512 columns
// of TMEM; calls with few such tiles take 128 or 64 columns (plan_fp8_gemm).
// The accumulators swap roles from tile to tile: tile i sums into region i & 1
// and its rank-r term goes to the other region, just before the tile's last
// blocks, when the epilogue has drained tile i - 1 from there; the epilogue
// moves the rank-r term into registers while those last blocks run, which
// frees that region for tile i + 1.  So the tensor pipe waits for no epilogue
// on long contractions.
//
// A product with few tiles is cut along its contraction: the pairs of a cluster
// share a tile and add their sums over distributed shared memory in rank order.
//
// Per CTA (384 threads):
//   warp 0      TMA producer, three stages of two blocks (64 KB); both CTAs'
//               copies complete on the leader's barrier
//   warp 1      TMEM allocation; in the leader CTA, this warp issues every MMA
//   warps 2, 3  scales of A and B: four blocks at a time into the MMA's layout
//               (32 lanes x 16 bytes per 128 rows), copied to TMEM by the
//               MMA warp (tcgen05.cp, replicated to the four lane quarters)
//   warps 4-11  epilogue: four lane quarters x two column halves
#include <algorithm>
#include <atomic>

#include "wl_common.cuh"
#include "wl_fp8.h"
#include "wl_fp8_device.cuh"

namespace wl {

namespace {

constexpr uint32_t kABytes = 16384;
constexpr int kLrLead = 2;           // main stages issued after the rank-r blocks
constexpr int kStoreStride = 18;     // bf16 of a staged row of 16 outputs (nine banks apart)
constexpr int kStoreBytes = 32 * kStoreStride * 2;  // per epilogue warp

// ------------------------------------------------------ CTA-pair primitives ----
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tmap, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_mxf8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
// 32 rows x 16 bytes of shared memory into four TMEM columns of every lane quarter.
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the tcgen05
// operations issued so far have ended.
__device__ __forceinline__ void commit_pair(uint64_t *bar, uint16_t pair_mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(pair_mask)
        : "memory");
}

// N-major tile of `bytes` (128, 64 or 32) columns x 128 contraction rows, as
// TMA leaves it with the swizzle of that width (modes 2, 4, 6): eight rows are
// 8 * bytes apart.
__device__ __forceinline__ uint64_t n_major_desc(uint32_t addr, uint32_t bytes) {
    const uint64_t mode = bytes == 128 ? 2 : bytes == 64 ? 4 : 6;
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(8 * bytes >> 4) << 32 | (uint64_t)1 << 46 |
           mode << 61;
}

// ---------------------------------------------------------------- schedule ----
struct Tile {
    int out, m0, n0;
};
__device__ __forceinline__ Tile tile_of(const Fp8GemmParams &p, int t) {
    t /= p.ranges;
    int o = 0;
    while (o + 1 < p.nout && t >= p.out[o + 1].tile_begin) ++o;
    const int local = t - p.out[o].tile_begin;
    return {o, (local % p.m_tiles) * kFp8BM, (local / p.m_tiles) * p.BN};
}

// The stages that a pair runs, and the one before which the rank-r blocks come.
struct Stages {
    int begin, end, low_at;
};

// Piece `pair` of p.split, or, for tile t of a product summed in ranges, its range.
__device__ __forceinline__ Stages stages_of(const Fp8GemmParams &p, const Fp8Out &o, int pair, int t) {
    int total = 0;
    for (int q = 0; q < o.nparts; ++q) total += (p.part[o.part0 + q].nkb + 1) >> 1;
    Stages r;
    const int piece = p.ranges > 1 ? t % p.ranges : pair, pieces = p.ranges > 1 ? p.ranges : p.split;
    r.begin = total * piece / pieces;
    r.end = total * (piece + 1) / pieces;
    r.low_at = pair == p.split - 1 ? max(r.begin, total - kLrLead) : -1;  // with the last range
    return r;
}

// A tile's work in issue order, up to two blocks (one stage) at a time:
// main(part, block, two) part by part, and before the last kLrLead stages of
// them low(part, block, two) for the rank-r blocks of every part.  Stops when
// either returns false.  The issuing warp's instructions bound how fast the
// tensor pipe is fed: an MMA takes it about 40 cycles, a barrier wait 70 and a
// commit 46, against 448 cycles of MMAs per block, so a stage holds two blocks
// and the order is in the loops, not in per-block state (with both per block a
// block took 950 cycles).
template <typename Main, typename Low>
__device__ __forceinline__ bool for_stages(const Fp8GemmParams &p, const Fp8Out &o, const Stages &r, Main main, Low low) {
    int i = 0;
    for (int q = o.part0; q < o.part0 + o.nparts && i < r.end; ++q) {
        const int nkb = p.part[q].nkb;
        int kb = 0;
        if (i < r.begin) {  // skip to the range
            const int skip = min(r.begin - i, (nkb + 1) >> 1);
            i += skip;
            kb = 2 * skip;
        }
        for (; kb < nkb && i < r.end; kb += 2, ++i) {
            if (i == r.low_at) {
                for (int l = o.part0; l < o.part0 + o.nparts; ++l) {
                    const int lr = p.part[l].lr;
                    for (int j = 0; j < lr; j += 2)
                        if (!low(l, j, j + 1 < lr)) return false;
                }
            }
            if (!main(q, kb, kb + 1 < nkb)) return false;
        }
    }
    return true;
}

__device__ __forceinline__ int lr_blocks(const Fp8GemmParams &p, const Fp8Out &o) {
    int lr = 0;
    for (int q = 0; q < o.nparts; ++q) lr += p.part[o.part0 + q].lr;
    return lr;
}

// The scale words of one chunk of B for output columns n0 .. n0 + 255.
template <bool kT>
__device__ __forceinline__ void b_scale_words(const Fp8Part &pt, int N, int n0, int q, int lane, uint32_t (&w)[8]) {
    if (!kT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = n0 + i * 32 + lane;
            w[i] = n < N ? __ldg(reinterpret_cast<const uint32_t *>(pt.b_scales + (size_t)(n >> 7) * pt.b_pitch + 4 * q))
                         : 0x7F7F7F7Fu;
        }
    } else {
        // byte i of a word: contraction block 4q + i; 256 columns touch at most three blocks of columns
        const int c0 = n0 >> 7, blk = lane >> 2, i = lane & 3;
        uint32_t b = 0x7Fu;
        if (blk < 3 && (c0 + blk) * 128 < N && 4 * q + i < pt.nkb)
            b = __ldg(pt.b_scales + (size_t)(4 * q + i) * pt.b_pitch + c0 + blk);
        b <<= 8 * i;
        b |= __shfl_xor_sync(0xffffffffu, b, 1);
        b |= __shfl_xor_sync(0xffffffffu, b, 2);
        const uint32_t w0 = __shfl_sync(0xffffffffu, b, 0), w1 = __shfl_sync(0xffffffffu, b, 4),
                       w2 = __shfl_sync(0xffffffffu, b, 8);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = ((n0 + k * 32 + lane) >> 7) - c0;
            w[k] = c == 0 ? w0 : c == 1 ? w1 : w2;
        }
    }
}

}  // namespace

template <int kMode, int kBN>
__global__ void __launch_bounds__(kFp8GemmThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
    constexpr bool kT = kMode == kFp8Transposed;
    constexpr int kHalf = kBN / 2;  // columns per CTA's half of B, and per epilogue warp
    constexpr int kChunks = kHalf / 16;
    constexpr uint32_t kRow = kHalf > 64 ? 128 : kHalf;  // bytes of a row of N-major B
    constexpr uint32_t kUBytes = kHalf * 128, kBBytes = kT ? kRow * 128 : kUBytes;
    constexpr uint32_t kRegionCols = kBN;  // region r at columns r * kBN
    constexpr uint32_t kSfCol = 2 * kBN;   // two slots of scales, 16 columns apart: A (4 columns), B (8)
    if (p.early_next) pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sf_base = base + kFp8Stages * kFp8StageBytes;
    uint8_t *store_base = sf_base + kFp8SfSlots * kFp8SfBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(store_base + 8 * kStoreBytes);
    uint64_t *empty = full + kFp8Stages;
    uint64_t *sf_full = empty + kFp8Stages;
    uint64_t *sf_empty = sf_full + kFp8SfSlots;
    uint64_t *m_full = sf_empty + kFp8SfSlots;  // [2] main sum of a region complete
    uint64_t *m_empty = m_full + 2;             // [2] ... and drained
    uint64_t *l_full = m_empty + 2;             // rank-r term complete
    uint64_t *l_empty = l_full + 1;             // ... and drained
    uint64_t *drain = l_empty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const WaitLimits limits{p.status, p.timeout_ns, abort_flag};

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA in its pair, its pair in the cluster
    const uint32_t rank = cluster_ctarank() & 1u, leader = cluster_ctarank() & ~1u;
    const int pair = (int)(leader >> 1);
    const uint16_t pair_mask = (uint16_t)(3u << leader);
    const int cluster = blockIdx.x / (2 * p.split), nclusters = gridDim.x / (2 * p.split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kFp8Stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kFp8SfSlots; ++i) {
            mbar_init(&sf_full[i], 4);  // two warps of each CTA
            mbar_init(&sf_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m_full[i], 1);
            mbar_init(&m_empty[i], 16);  // eight warps of each CTA
        }
        mbar_init(l_full, 1);
        mbar_init(l_empty, 16);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_primary();

    if (warp == 0) {
        // ------------------------------------------------------ producer ----
        Ring r(kFp8Stages);
        uint32_t issued = 0;
        const uint32_t stage0 = smem_addr(base), full0 = map_rank(full, leader);
        bool ok = true;
        for (int t = cluster; t < p.num_tiles && ok; t += nclusters) {
            const Tile ti = tile_of(p, t);
            const int m = ti.m0 + (int)rank * 128, n = ti.n0 + (int)rank * kHalf;
            // one or two blocks of `step` columns into the next stage; both CTAs'
            // bytes are expected by the leader
            auto load = [&](const CUtensorMap *ma, const CUtensorMap *mb, int c, int step, bool two, bool rows_of_b, uint32_t b_bytes) {
                if (!warp_wait(&empty[r.slot], r.phase ^ 1u, limits)) return false;
                if (elect_one()) {
                    const uint32_t bar = full0 + r.slot * 8;
                    uint32_t sa = stage0 + r.slot * kFp8StageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[r.slot], (2 * (kABytes + b_bytes)) << two);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k == 1 && !two) break;
                        tma_load_2d_pair(sa, ma, c, m, bar);
                        tma_load_2d_pair(sa + kABytes, mb, rows_of_b ? n : c, rows_of_b ? c : n, bar);
                        c += step;
                        sa += kFp8BlockBytes;
                    }
                }
                __syncwarp();
                r.advance();
                ++issued;
                return true;
            };
            const Fp8Out &o = p.out[ti.out];
            ok = for_stages(
                p, o, stages_of(p, o, pair, t),
                [&](int q, int kb, bool two) { return load(&p.tm_a[q], &p.tm_b[q], kb * 128, 128, two, kT, kBBytes); },
                [&](int q, int j, bool two) { return load(&p.tm_t[q], &p.tm_u[q], j * 64, 64, two, false, kUBytes); });
        }
        if (!ok && lane == 0) {
            // Let the copies already issued land before the pair exits.  Their
            // bytes are counted in the leader; the other CTA gives its own time.
            if (rank == 0) {
                const uint32_t left = issued < kFp8Stages ? issued : kFp8Stages;
                for (uint32_t i = issued - left; i < issued; ++i)
                    mbar_wait(&full[i % kFp8Stages], (i / kFp8Stages) & 1u, p.status, 1000000ull);
            } else {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer ---
        if (rank == 0) {
            const uint32_t idesc_lr = idesc_bf16_f32(kFp8BM, kBN), idesc0 = idesc_mxf8(kFp8BM, kBN, kT);
            const uint32_t sb = smem_addr(base) + kABytes;
            const uint64_t da0 = sw128_kmajor_desc(smem_addr(base)), du0 = sw128_kmajor_desc(sb);
            const uint64_t db0 = kT ? n_major_desc(sb, kRow) : du0;
            const uint64_t sd0 = scale_desc(smem_addr(sf_base));
            constexpr uint64_t kNext = kFp8BlockBytes >> 4;  // a stage's second block
            // 32 columns of the contraction further: 32 bytes inside the swizzled
            // rows, or (N-major) 32 rows
            constexpr uint64_t kStepB = kT ? 2 * kRow : 2;
            Ring r(kFp8Stages), sr(kFp8SfSlots);
            uint32_t it = 0, lr_count = 0, sf_slot = 0;
            bool ok = true;
            for (int t = cluster; t < p.num_tiles && ok; t += nclusters, ++it) {
                const Tile ti = tile_of(p, t);
                const Fp8Out &o = p.out[ti.out];
                const uint32_t reg = it & 1u, other = reg ^ 1u;
                const uint32_t d_main = tmem + reg * kRegionCols, d_lr = tmem + other * kRegionCols;
                const uint32_t uses = it >> 1, other_uses = (it + 1) >> 1;  // of the regions, by earlier tiles
                // the region's last main sum and the last rank-r term have been read
                if (uses > 0) ok = warp_wait<true>(&m_empty[reg], (uses - 1) & 1u, limits);
                if (ok && lr_count > 0) ok = warp_wait<true>(l_empty, (lr_count - 1) & 1u, limits);
                if (!ok) break;
                tc_fence_after();
                const Stages range = stages_of(p, o, pair, t);
                const int lr = range.low_at >= 0 ? lr_blocks(p, o) : 0;
                int lr_left = lr;
                uint32_t acc = 0;
                ok = for_stages(
                    p, o, range,
                    [&](int, int kb, bool two) {
                        const bool chunk = (kb & 3) == 0 || acc == 0;  // the next four blocks' scales
                        if (chunk) {
                            if (!warp_wait<true>(&sf_full[sr.slot], sr.phase, limits)) return false;
                            sf_slot ^= 16u;
                        }
                        if (!warp_wait(&full[r.slot], r.phase, limits)) return false;
                        tc_fence_after();
                        const uint32_t sf = tmem + kSfCol + sf_slot, idesc = idesc0 + (kb & 3) * kScaleByte;
                        const uint64_t da = da0 + r.slot * (kFp8StageBytes >> 4), db = db0 + r.slot * (kFp8StageBytes >> 4);
                        const uint64_t ds = sd0 + sr.slot * (kFp8SfBytes >> 4);
                        if (elect_one()) {
                            if (chunk) {
                                cp_scales_pair(sf, ds);
                                cp_scales_pair(sf + 4, ds + (512 >> 4));
                                if (kBN > 128) cp_scales_pair(sf + 8, ds + (1024 >> 4));
                                commit_pair(&sf_empty[sr.slot], pair_mask);
                            }
                            mma_mxf8_pair(d_main, da, db, idesc, sf, sf + 4, acc);
#pragma unroll
                            for (int k = 1; k < 4; ++k) mma_mxf8_pair(d_main, da + 2 * k, db + kStepB * k, idesc, sf, sf + 4, 1);
                            if (two)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_mxf8_pair(d_main, da + kNext + 2 * k, db + kNext + kStepB * k, idesc + kScaleByte, sf, sf + 4, 1);
                            commit_pair(&empty[r.slot], pair_mask);
                        }
                        __syncwarp();
                        acc = 1;
                        if (chunk) sr.advance();
                        r.advance();
                        return true;
                    },
                    [&](int, int, bool two) {
                        const bool first = lr_left == lr;
                        if (first && other_uses > 0 && !warp_wait<true>(&m_empty[other], (other_uses - 1) & 1u, limits)) return false;
                        if (!warp_wait(&full[r.slot], r.phase, limits)) return false;
                        tc_fence_after();
                        lr_left -= 1 + two;
                        const uint64_t da = da0 + r.slot * (kFp8StageBytes >> 4), db = du0 + r.slot * (kFp8StageBytes >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) mma_f16_pair(d_lr, da + 2 * k, db + 2 * k, idesc_lr, !(first && k == 0));
                            if (two)
#pragma unroll
                                for (int k = 0; k < 4; ++k) mma_f16_pair(d_lr, da + kNext + 2 * k, db + kNext + 2 * k, idesc_lr, 1);
                            commit_pair(&empty[r.slot], pair_mask);
                            if (lr_left == 0) commit_pair(l_full, pair_mask);
                        }
                        __syncwarp();
                        r.advance();
                        return true;
                    });
                if (!ok) break;
                if (elect_one()) commit_pair(&m_full[reg], pair_mask);
                __syncwarp();
                lr_count += lr > 0;
            }
            if (elect_one()) commit_pair(drain, pair_mask);
            __syncwarp();
        }
    } else if (warp < 4) {
        // ------------------------------------------------------- scales -----
        Ring r(kFp8SfSlots);
        bool ok = true;
        for (int t = cluster; t < p.num_tiles && ok; t += nclusters) {
            const Tile ti = tile_of(p, t);
            const Fp8Out &o = p.out[ti.out];
            const Stages range = stages_of(p, o, pair, t);
            for (int q = 0, i = 0; q < o.nparts && ok; ++q) {
                const Fp8Part &pt = p.part[o.part0 + q];
                // stages i + 2c and i + 2c + 1 take chunk c
                const int stages = (pt.nkb + 1) >> 1, first = max(range.begin - i, 0), last = min(range.end - i, stages);
                i += stages;
                for (int c = first >> 1; first < last && 2 * c < last; ++c) {
                    uint32_t w[8];
                    if (warp == 2) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int m = ti.m0 + (int)rank * 128 + i * 32 + lane;
                            w[i] = m < p.M ? __ldg(reinterpret_cast<const uint32_t *>(pt.a_scales + (size_t)m * pt.a_pitch + 4 * c))
                                           : 0x7F7F7F7Fu;
                        }
                    } else {
                        b_scale_words<kT>(pt, o.N, ti.n0, c, lane, w);
                    }
                    if (!warp_wait(&sf_empty[r.slot], r.phase ^ 1u, limits)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = sf_base + r.slot * kFp8SfBytes + lane * 16;
                    if (warp == 2) {
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        *reinterpret_cast<uint4 *>(dst + 512) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4 *>(dst + 1024) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) arrive_cluster(map_rank(&sf_full[r.slot], leader));
                    r.advance();
                }
            }
        }
    } else {
        // ------------------------------------------------------- epilogue ---
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16) + half * kHalf;
        const uint32_t m_empty_l = map_rank(m_empty, leader);
        const uint32_t l_empty_l = map_rank(l_empty, leader);
        uint32_t it = 0, lr_count = 0;
        for (int t = cluster; t < p.num_tiles; t += nclusters, ++it) {
            const Tile ti = tile_of(p, t);
            const Fp8Out &o = p.out[ti.out];
            const uint32_t reg = it & 1u;
            const int lr = pair == p.split - 1 ? lr_blocks(p, o) : 0;
            const int m = ti.m0 + (int)rank * 128 + quarter * 32 + lane;
            const int n0 = ti.n0 + half * kHalf;
            uint32_t d[kChunks][16];
            if (kMode != kFp8ColSums && lr > 0) {
                if (!warp_wait(l_full, lr_count & 1u, limits)) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kChunks; ++c) tmem_ld16(lane_addr + (reg ^ 1u) * kRegionCols + c * 16, d[c]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(l_empty_l);
                ++lr_count;
            } else {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) d[c][i] = 0;
            }
            if (!warp_wait(&m_full[reg], (it >> 1) & 1u, limits)) break;
            tc_fence_after();
            if (kMode == kFp8ColSums) {
                const bool vec = (o.N & 7) == 0 && (reinterpret_cast<uintptr_t>(o.dy) & 15u) == 0;
                const __nv_bfloat16 *dyr = o.dy + (size_t)m * o.N;
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    const int n = n0 + c * 16;
                    uint32_t v[16];
                    tmem_ld16(lane_addr + reg * kRegionCols + c * 16, v);
                    float g[16];
                    if (m < p.M && vec && n + 16 <= o.N) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(dyr + n), b = *reinterpret_cast<const uint4 *>(dyr + n + 8);
                        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            g[2 * i] = bf16lo(w[i]);
                            g[2 * i + 1] = bf16hi(w[i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) g[i] = m < p.M && n + i < o.N ? __bfloat162float(dyr[n + i]) : 0.f;
                    }
                    tmem_ld_wait();
                    // rows that do not exist add nothing, whatever their accumulator holds
#pragma unroll
                    for (int i = 0; i < 16; ++i) g[i] = m < p.M ? g[i] * __uint_as_float(v[i]) : 0.f;
                    // transpose-and-add over the 32 rows: lane l ends with column l & 15
#pragma unroll
                    for (int w = 8; w > 0; w >>= 1) {
                        const bool up = lane & w;
#pragma unroll
                        for (int i = 0; i < w; ++i) {
                            const float send = up ? g[i] : g[i + w], keep = up ? g[i + w] : g[i];
                            g[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                        }
                    }
                    g[0] += __shfl_xor_sync(0xffffffffu, g[0], 16);
                    const int row = (ti.m0 >> 5) + (int)rank * 4 + quarter;
                    if (lane < 16 && n + lane < o.N && row * 32 < p.M)
                        o.sums[((size_t)(t % p.ranges) * ((p.M + 31) >> 5) + row) * o.N + n + lane] = g[0];
                }
            } else {
                const bool vec = (o.N & 7) == 0 && (reinterpret_cast<uintptr_t>(o.y) & 15u) == 0;
                const bool svec = (reinterpret_cast<uintptr_t>(o.s) & 15u) == 0;
                __nv_bfloat16 *yr = o.y + (size_t)m * o.N;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int n = n0 + c * 16;
                    uint32_t v[16];
                    tmem_ld16(lane_addr + reg * kRegionCols + c * 16, v);
                    float sc[16];
                    if (o.s && svec && n + 16 <= o.N) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 f = __ldg(reinterpret_cast<const float4 *>(o.s + n) + i);
                            sc[4 * i] = f.x;
                            sc[4 * i + 1] = f.y;
                            sc[4 * i + 2] = f.z;
                            sc[4 * i + 3] = f.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) sc[i] = o.s && n + i < o.N ? __ldg(o.s + n + i) : 1.f;
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) sc[i] = fmaf(sc[i], __uint_as_float(v[i]), __uint_as_float(d[c][i]));
                    if (p.split > 1) {  // into the idle stages, [column][row]
                        float *sums = reinterpret_cast<float *>(base) + (half * kHalf + c * 16) * 128 + quarter * 32 + lane;
#pragma unroll
                        for (int i = 0; i < 16; ++i) sums[i * 128] = sc[i];
                        continue;
                    }
                    if (m < p.M) {
                        if (vec && n + 16 <= o.N) {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                *reinterpret_cast<uint4 *>(yr + n + 8 * i) =
                                    make_uint4(pack_bf16x2(sc[8 * i], sc[8 * i + 1]), pack_bf16x2(sc[8 * i + 2], sc[8 * i + 3]),
                                               pack_bf16x2(sc[8 * i + 4], sc[8 * i + 5]), pack_bf16x2(sc[8 * i + 6], sc[8 * i + 7]));
                        }
                    }
                    if (!vec || n + 16 > o.N) {
                        // rows that are not 16-byte aligned: 16 lanes per row
                        __nv_bfloat16 *buf = reinterpret_cast<__nv_bfloat16 *>(store_base + (warp - 4) * kStoreBytes);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<uint32_t *>(buf + lane * kStoreStride)[i] = pack_bf16x2(sc[2 * i], sc[2 * i + 1]);
                        __syncwarp();
                        const int col = lane & 15;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const int row = i + (lane >> 4), mr = m - lane + row;
                            if (mr < p.M && n + col < o.N) o.y[(size_t)mr * o.N + n + col] = buf[row * kStoreStride + col];
                        }
                        __syncwarp();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(m_empty_l + reg * 8);
        }
    }

    if (kMode != kFp8ColSums && p.split > 1) {
        __syncwarp();
        cluster_sync();  // every pair's sums are in its shared memory
        if (warp >= 4) {
            // groups of 16 columns go round the pairs; a thread adds eight columns of a row
            const Tile ti = tile_of(p, cluster);
            const Fp8Out &o = p.out[ti.out];
            const int tid = threadIdx.x - 128, row = tid & 127, m = ti.m0 + (int)rank * 128 + row;
            const bool vec = (o.N & 7) == 0 && (reinterpret_cast<uintptr_t>(o.y) & 15u) == 0;
            for (int g = pair; g < kBN / 16; g += p.split) {
                const int c = g * 16 + (tid >> 7) * 8, n = ti.n0 + c;
                const float *sums = reinterpret_cast<const float *>(base) + c * 128 + row;
                float v[8] = {};
#pragma unroll 2
                for (int s = 0; s < p.split; ++s) {
                    float a[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = ld_cluster(sums + i * 128, 2 * s + rank);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += a[i];
                }
                if (m >= p.M) continue;
                __nv_bfloat16 *y = o.y + (size_t)m * o.N + n;
                if (vec && n + 8 <= o.N) {
                    *reinterpret_cast<uint4 *>(y) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (n + i < o.N) y[i] = __float2bfloat16_rn(v[i]);
                }
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // Every MMA issued has ended and every signal of theirs has arrived here.
    if (warp == 1) mbar_wait(drain, 0, p.status, kDrainNs);
    cluster_sync();  // no CTA leaves while another may signal it, its MMAs read there or its sums are read
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

namespace {
constexpr size_t kGemmSmem = 1024 + kFp8Stages * kFp8StageBytes + kFp8SfSlots * kFp8SfBytes + 8 * kStoreBytes +
                             (2 * kFp8Stages + 2 * kFp8SfSlots + 7) * 8 + 16;
static_assert(kGemmSmem <= 227 * 1024, "shared memory of one CTA");

using GemmKernel = void (*)(Fp8GemmParams);
template <int kMode>
GemmKernel kernel_of(int bn) {
    return bn == 224 ? fp8_gemm_kernel<kMode, 224> : bn == 128 ? fp8_gemm_kernel<kMode, 128> : fp8_gemm_kernel<kMode, 64>;
}
}  // namespace

// The tile width and cut with the least estimated cycles: waves of tiles over
// the CTA pairs, a block of the contraction at the slowest of the MMAs (2 cycles
// per column), the loads (kFp8GemmFill) and the issue (330 cycles), about
// 5000 cycles to start and drain a tile, and for a cut tile, all pairs of whose
// clusters have to be resident, 3000 and 25 per column for the exchange.
// 512 x 1152 over 8192: 12 whole tiles of 224 columns take 37 us.
void plan_fp8_gemm(Fp8GemmParams &p, const int *N, int nout, int blocks, bool may_split, int num_sms) {
    // clusters of 1, 2, .. 8 pairs that a B200 holds at once
    static const int kResident[8] = {74, 33, 22, 15, 11, 7, 7, 7};
    const int m_tiles = (p.M + kFp8BM - 1) / kFp8BM, pairs = num_sms / 2;
    double least = 0;
    for (int bn : {224, 128, 64}) {
        long long tiles = 0;
        for (int i = 0; i < nout; ++i) tiles += (long long)m_tiles * ((N[i] + bn - 1) / bn);
        const double block = std::max({2.0 * bn, (16384 + 64.0 * bn) / kFp8GemmFill, 330.0});
        for (int s = 1; s <= 8; ++s) {
            if (s > 1 && (!may_split || tiles > kResident[s - 1] || blocks < 4 * s)) break;
            const double cost = (double)((tiles + pairs - 1) / pairs) * ((blocks + s - 1) / s * block + 5000) +
                                (s > 1 ? 3000 + 25.0 * bn : 0);
            if (least == 0 || cost < least) {
                least = cost;
                p.BN = bn;
                p.split = s;
            }
        }
    }
    p.m_tiles = m_tiles;
    p.ranges = 1;
}

cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, Fp8Mode mode, int num_sms, cudaStream_t stream) {
    if (p.num_tiles == 0) return cudaSuccess;
    const GemmKernel kernel = mode == kFp8Plain ? kernel_of<kFp8Plain>(p.BN)
                              : mode == kFp8Transposed ? kernel_of<kFp8Transposed>(p.BN) : kernel_of<kFp8ColSums>(p.BN);
    // Opt in to the large shared-memory carve-out once per device and kernel.
    static std::atomic<bool> done[64][3][3] = {};
    const int width = p.BN == 224 ? 0 : p.BN == 128 ? 1 : 2;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev][mode][width].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGemmSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done[dev][mode][width].store(true, std::memory_order_release);
    }
    if (p.ranges > 1 && mode != kFp8ColSums) return cudaErrorInvalidValue;
    // a cut tile has a cluster of its own
    const int clusters = p.split == 1 && num_sms / 2 < p.num_tiles ? num_sms / 2 : p.num_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.split * clusters);
    cfg.blockDim = dim3(kFp8GemmThreads);
    cfg.dynamicSmemBytes = kGemmSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

namespace {
// 32 columns x 32 partial sums per step and CTA, so a warp reads 128 bytes of
// a row; each thread adds every 32nd row, then the 32 sums of a column meet in
// a fixed order.
__global__ void __launch_bounds__(1024) sum_rows_kernel(const __grid_constant__ Fp8SumParams p) {
    __shared__ float part[32][33];
    pdl_wait_primary();
    pdl_launch_dependents();
    int jx = 0;
    while (jx + 1 < p.njobs && (int)blockIdx.x >= p.job[jx + 1].cta_begin) ++jx;
    const Fp8SumJob &jb = p.job[jx];
    const int n0 = ((int)blockIdx.x - jb.cta_begin) * 32, n = n0 + threadIdx.x;
    float a = 0.f;
    if (n < jb.N)
        for (int i = threadIdx.y; i < p.n_rows; i += 32) a += jb.sums[(size_t)i * jb.N + n];
    part[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    const float v = warp_sum(part[threadIdx.x][threadIdx.y]);
    const int m = n0 + threadIdx.y;
    if (threadIdx.x == 0 && m < jb.N) jb.ds[m] = v;
}
}  // namespace

cudaError_t launch_fp8_sum_rows(Fp8SumParams &p, cudaStream_t stream) {
    int ctas = 0;
    for (int i = 0; i < p.njobs; ++i) {
        p.job[i].cta_begin = ctas;
        ctas += (p.job[i].N + 31) / 32;
    }
    if (ctas == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_rows_kernel, p);
}

}  // namespace wl
