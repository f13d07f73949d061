// What the 8-bit tensor-core kernels share: bounded waits and elections of
// warps that issue copies and MMAs, scale descriptors, TMEM loads.
//
// A warp that issues runs its loops whole and elects one lane for the issue
// alone: in warp-uniform code the operands sit in uniform registers, and a
// stage of four MMAs with its wait and commit takes the warp 281 cycles to
// issue, against 446 when a single thread runs the loop.
#pragma once

#include "wl_common.cuh"

namespace wl {

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

// Like mbar_try_wait, for barriers that the cluster's other CTA arrives on.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster; whole warps arrive together.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// shared::cluster address of `p` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
// The float at `p` in the CTA `rank`.
__device__ __forceinline__ float ld_cluster(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_rank(p, rank)) : "memory");
    return v;
}

// TMEM and kernels that share an SM: an allocation waits until there is room,
// so a CTA that holds TMEM must never wait for another CTA or kernel.  The
// kernels that leave room for a neighbour therefore allocate after their wait
// for the previous kernel (which may itself be waiting for TMEM) and release
// before they meet the other CTAs of their cluster.

// What a kernel's waits need: where errors go, when to give up, and a flag in
// shared memory by which one warp's time-out stops the others.
struct WaitLimits {
    int *status;
    uint64_t timeout_ns;
    volatile int *abort_flag;
};

// A whole warp waits for a phase of `bar`; the lanes go on, or give up, together.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const WaitLimits &w) {
    bool done = kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (!done) done = kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, done)) return true;
        const bool late = globaltimer_ns() - t0 > w.timeout_ns;
        if (__any_sync(0xffffffffu, late || *w.abort_flag != 0)) {
            if (late) record_status(w.status, kStatusTimeout);
            if ((threadIdx.x & 31) == 0) *w.abort_flag = 1;
            return false;
        }
    }
}

// Bound on the wait for MMAs already issued: they end by themselves, whatever
// limit the other waits have, and TMEM must not be released before.
constexpr uint64_t kDrainNs = 10000000;

// Scales of 128 rows in shared memory (32 x 16 bytes, unswizzled, 8-row groups
// 128 bytes apart), for the copy to TMEM.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// Instruction descriptor of kind::mxf8f6f4: E4M3 A and B (formats 0), E8M0
// scales (bit 23), N >> 3 (17-22), M >> 7 (27-28), the byte of the scale words
// (4-5 for B, 29-30 for A; adding kScaleByte takes the next); bit 16: B N-major.
constexpr uint32_t kScaleByte = (1u << 4) | (1u << 29);
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, bool b_n_major = false) {
    return (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// Position in a ring of n slots.
struct Ring {
    uint32_t slot = 0, phase = 0, n;
    __device__ explicit Ring(uint32_t n_) : n(n_) {}
    __device__ void advance() {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

}  // namespace wl
