// C ABI of the 8-bit operators: argument checks, the workspace's layout and
// the order of the launches.  Contracts in include/wl.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <memory>
#include <new>

#include "../../include/wl.h"
#include "wl_fp8.h"

namespace wl {

namespace {

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
wl_status from_cuda(cudaError_t e) { return e == cudaSuccess ? WL_OK : WL_ERR_CUDA; }
long long round16(long long v) { return (v + 15) & ~15LL; }

// Hands out 256-byte-aligned parts of a workspace; with no base it only counts.
struct Arena {
    uint8_t *base;
    size_t used = 0;
    explicit Arena(void *p) : base(static_cast<uint8_t *>(p)) {}
    template <typename T>
    T *take(size_t n) {
        const size_t at = used;
        used += (n * sizeof(T) + 255) & ~size_t(255);
        return base ? reinterpret_cast<T *>(base + at) : nullptr;
    }
};

constexpr int kWsAlign = 16;
constexpr int kMaxSize = 1 << 30;  // rows or columns: indexes past them still fit an int

wl_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return WL_OK;
    if (!ws || have < need) return WL_ERR_INVALID_ARG;
    return aligned(ws, kWsAlign) ? WL_OK : WL_ERR_ALIGNMENT;
}

// ---------------------------------------------------------------- forward ----
template <typename Proj>
wl_status check_sizes(int M, int K, const Proj *projs, int P) {
    if (!projs) return WL_ERR_INVALID_ARG;
    if (P < 1) return WL_ERR_INVALID_ARG;
    if (P > WL_MAX_PROJ) return WL_ERR_UNSUPPORTED;
    if (M < 0 || K < 0) return WL_ERR_INVALID_ARG;
    if (M > kMaxSize || K > kMaxSize) return WL_ERR_UNSUPPORTED;
    for (int i = 0; i < P; ++i) {
        if (projs[i].N < 0 || projs[i].r < 0) return WL_ERR_INVALID_ARG;
        if (projs[i].r > WL_MAX_RANK || projs[i].N > kMaxSize) return WL_ERR_UNSUPPORTED;
    }
    if (K % 16 != 0) return WL_ERR_ALIGNMENT;
    for (int i = 0; i < P; ++i)
        if (projs[i].r % 8 != 0) return WL_ERR_ALIGNMENT;
    return WL_OK;
}

// The few-token kernel's cut of a product; s, y, maps and pointers are not set.
void plan_stream(Fp8StreamParams &sp, int M, int K, const int *N, const int *r, int P) {
    std::memset(&sp, 0, sizeof sp);
    sp.M = M;
    sp.pitch = fp8_pitch(K);
    for (int i = 0; i < P; ++i) {
        if (N[i] == 0) continue;
        Fp8StreamSeg &sg = sp.seg[sp.nseg++];
        sg.N = N[i];
        sg.nkb = (K + kFp8Block - 1) / kFp8Block;
        sg.lr = (r[i] + 63) / 64;
    }
    plan_fp8_stream(sp);
}

struct ForwardLayout {
    uint8_t *codes, *scales;
    __nv_bfloat16 *T[kMaxSeg];
    float *parts;
    unsigned int *counters;
    size_t bytes;
};

// With projs->T set or not, and x_codes given or not, the layout is the same.
ForwardLayout forward_layout(int M, int K, const wl_proj_fp8 *projs, int P, void *ws) {
    ForwardLayout l = {};
    Arena a(ws);
    l.codes = a.take<uint8_t>((size_t)M * K);
    l.scales = a.take<uint8_t>((size_t)M * fp8_pitch(K));
    for (int i = 0; i < P; ++i) l.T[i] = a.take<__nv_bfloat16>((size_t)M * projs[i].r);
    if (M > 0 && M <= kFp8StreamMaxM && K > 0) {
        int N[kMaxSeg], r[kMaxSeg];
        for (int i = 0; i < P; ++i) N[i] = projs[i].N, r[i] = projs[i].r;
        Fp8StreamParams sp;
        plan_stream(sp, M, K, N, r, P);
        l.parts = a.take<float>(fp8_stream_part_floats(sp));
        l.counters = a.take<unsigned int>(sp.tiles);
    }
    l.bytes = a.used;
    return l;
}

wl_status forward_check(const wl_bf16 *x, int M, int K, const wl_proj_fp8 *projs, int P, const uint8_t *x_codes,
                        const uint8_t *x_scales) {
    wl_status st = check_sizes(M, K, projs, P);
    const bool sizes_aligned = st != WL_ERR_ALIGNMENT;
    if (st != WL_OK && sizes_aligned) return st;
    if ((x_codes == nullptr) != (x_scales == nullptr)) return WL_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && !x) return WL_ERR_INVALID_ARG;
    for (int i = 0; i < P; ++i) {
        const wl_proj_fp8 &q = projs[i];
        if (M == 0) continue;
        if (q.N > 0 && (!q.y || !q.s || (K > 0 && (!q.codes || !q.scales)))) return WL_ERR_INVALID_ARG;
        if (q.r > 0 && K > 0 && (!q.V || (q.N > 0 && !q.U))) return WL_ERR_INVALID_ARG;
    }
    if (!sizes_aligned) return WL_ERR_ALIGNMENT;
    if (!aligned(x, 16) || !aligned(x_codes, 16) || !aligned(x_scales, 4)) return WL_ERR_ALIGNMENT;
    for (int i = 0; i < P; ++i) {
        const wl_proj_fp8 &q = projs[i];
        if (!aligned(q.codes, 16) || !aligned(q.scales, 4) || !aligned(q.s, 4) || !aligned(q.U, 16) ||
            !aligned(q.V, 16) || !aligned(q.T, 16) || !aligned(q.y, 2))
            return WL_ERR_ALIGNMENT;
    }
    return WL_OK;
}

// Tensor maps of one contraction part.  b_rows x b_cols: the codes of B as
// stored; lr_rows: rows of U (output columns of the product); same_a: A is the
// previous part's.
wl_status set_part(Fp8GemmParams &g, int i, const Fp8Mat &A, int M, int a_cols, const Fp8Mat &B, int b_rows, int b_cols,
                   bool transposed, const __nv_bfloat16 *T, const __nv_bfloat16 *U, int r, int lr_rows, bool same_a = false) {
    Fp8Part &pt = g.part[i];
    pt.a_scales = A.scales;
    pt.a_pitch = A.pitch;
    pt.b_scales = B.scales;
    pt.b_pitch = B.pitch;
    pt.nkb = (a_cols + kFp8Block - 1) / kFp8Block;
    pt.lr = (r + 63) / 64;
    wl_status st = WL_OK;
    if (same_a)
        g.tm_a[i] = g.tm_a[i - 1];
    else
        st = encode_map_2d_u8(&g.tm_a[i], A.codes, a_cols, M, A.ld, 128, 128);
    if (st == WL_OK) st = encode_map_2d_u8(&g.tm_b[i], B.codes, b_cols, b_rows, B.ld, transposed ? (g.BN > 128 ? 128 : g.BN / 2) : 128,
                                           transposed ? 128 : g.BN / 2);
    if (st == WL_OK && r > 0) st = encode_map_2d(&g.tm_t[i], T, r, M, r, 64, 128);
    if (st == WL_OK && r > 0) st = encode_map_2d(&g.tm_u[i], U, r, lr_rows, r, 64, g.BN / 2);
    return st;
}

Fp8Out &add_out(Fp8GemmParams &g, int N, int part0, int nparts) {
    Fp8Out &o = g.out[g.nout++];
    o.N = N;
    o.part0 = part0;
    o.nparts = nparts;
    o.tile_begin = g.num_tiles;
    g.num_tiles += g.m_tiles * ((N + g.BN - 1) / g.BN);  // times g.ranges, in the end
    return o;
}

const __nv_bfloat16 *bf16(const wl_bf16 *p) { return reinterpret_cast<const __nv_bfloat16 *>(p); }
__nv_bfloat16 *bf16(wl_bf16 *p) { return reinterpret_cast<__nv_bfloat16 *>(p); }

struct Device {
    int sms;
    int *status;
};

// Outputs of M rows x N[0..nout) columns over `blocks` blocks.
void init_gemm(Fp8GemmParams &g, int M, const int *N, int nout, int blocks, bool may_split, const Device &dev) {
    std::memset(&g, 0, sizeof g);
    g.M = M;
    plan_fp8_gemm(g, N, nout, blocks, may_split, dev.sms);
    g.early_next = true;
    g.status = dev.status;
    g.timeout_ns = wait_limit_ns();
}

void init_lowrank(LowrankParams &p, const Device &dev) {
    std::memset(&p, 0, sizeof p);
    p.status = dev.status;
    p.timeout_ns = wait_limit_ns();
}

// Adds out = A B (+ what its rounding left in out_low).  A: I x K (rows) or
// K x I (cols), rows lda elements apart; B: K x r.
wl_status add_lowrank(LowrankParams &p, LowrankMode mode, const __nv_bfloat16 *A, long long lda, int I, int K,
                      const __nv_bfloat16 *B, int r, __nv_bfloat16 *out, __nv_bfloat16 *out_low, bool same_a = false) {
    LowrankJob &j = p.job[p.njobs++];
    j.I = I;
    j.K = K;
    j.r = r;
    j.kb = (K + 63) / 64;
    j.out = out;
    j.out_low = out_low;
    // rows that do not exist need not be loaded: each fills its own row of the sums
    wl_status st = WL_OK;
    if (same_a)
        j.tm_a = p.job[p.njobs - 2].tm_a;
    else
        st = mode == kLowrankRows ? encode_map_2d(&j.tm_a, A, K, I, lda, 64, lowrank_a_rows(I))
                                  : encode_map_2d(&j.tm_a, A, I, K, lda, 64, 64);
    return st == WL_OK ? encode_map_2d(&j.tm_b, B, r, K, r, 64, 64) : st;
}

// Adds out = X^T (B + B_low) for X in 8 bits (K x I), the same for every job.
wl_status add_lowrank_codes(LowrankParams &p, const Fp8Mat &X, int I, int K, const __nv_bfloat16 *B,
                            const __nv_bfloat16 *B_low, int r, __nv_bfloat16 *out) {
    LowrankJob &j = p.job[p.njobs++];
    j.I = I;
    j.K = K;
    j.r = r;
    j.kb = (K + 63) / 64;
    j.a_scales = X.scales;
    j.a_pitch = X.pitch;
    j.out = out;
    wl_status st = WL_OK;
    if (p.njobs > 1)
        j.tm_a = p.job[0].tm_a;
    else
        st = encode_map_2d_u32(&j.tm_a, X.codes, I / 4, K, X.ld, 32, 64);
    if (st == WL_OK) st = encode_map_2d(&j.tm_b, B, r, K, r, 64, 64);
    return st == WL_OK ? encode_map_2d(&j.tm_b2, B_low, r, K, r, 64, 64) : st;
}

// The few-token kernel's parameters for y_p = s_p (.) (X W_p^T) + T_p U_p^T.
// parts and counters as plan_stream's cut needs them, counters zero at launch.
wl_status set_stream(Fp8StreamParams &sp, const Fp8Mat &X, int M, int K, const wl_proj_fp8 *projs,
                     __nv_bfloat16 *const *T, int P, float *parts, unsigned int *counters, bool early, const Device &dev) {
    int N[kMaxSeg], r[kMaxSeg];
    for (int i = 0; i < P; ++i) N[i] = projs[i].N, r[i] = projs[i].r;
    plan_stream(sp, M, K, N, r, P);
    sp.x_scales = X.scales;
    sp.early = early;
    sp.early_next = true;
    sp.parts = parts;
    sp.counters = counters;
    sp.status = dev.status;
    sp.timeout_ns = wait_limit_ns();
    wl_status st = encode_map_2d_u8(&sp.tm_x, X.codes, K, M, X.ld, 128, sp.Mp);
    int k = 0;
    for (int i = 0; i < P && st == WL_OK; ++i) {
        const wl_proj_fp8 &q = projs[i];
        if (q.N == 0) continue;
        sp.seg[k].w_scales = q.scales;
        sp.seg[k].s = q.s;
        sp.seg[k].y = bf16(q.y);
        st = encode_map_2d_u8(&sp.tm_w[k], q.codes, K, q.N, K, 128, 128);
        if (st == WL_OK && q.r > 0) st = encode_map_2d(&sp.tm_u[k], bf16(q.U), q.r, q.N, q.r, 64, 128);
        if (st == WL_OK && q.r > 0) st = encode_map_2d(&sp.tm_t[k], T[i], q.r, M, q.r, 64, sp.Mp);
        ++k;
    }
    return st;
}

}  // namespace
}  // namespace wl

// Everything a forward call launches.
struct wl_fp8_plan {
    int M, K, P;
    wl_proj_fp8 projs[WL_MAX_PROJ];
    bool zeros;                // K == 0: outputs are zero
    wl::Fp8RowsParams quant;   // njobs == 0: the rank-r launch quantises x, or nothing is to be done
    wl::LowrankParams lowrank;
    bool rows;                 // a short call: one launch
    wl::Fp8RowsForward short_call;
    bool few;                  // which of the two products otherwise
    wl::Fp8StreamParams stream;
    wl::Fp8GemmParams gemm;
};

namespace wl {
namespace {

// Sets `f` up for a checked call; launches nothing.
wl_status forward_plan(wl_fp8_plan &f, const wl_bf16 *x, int M, int K, const wl_proj_fp8 *projs, int P, uint8_t *x_codes,
                       uint8_t *x_scales, const ForwardLayout &l, const Device &dev) {
    f.M = M;
    f.K = K;
    f.P = P;
    f.quant.njobs = f.lowrank.njobs = f.stream.nseg = f.gemm.nout = 0;
    f.stream.units = f.gemm.num_tiles = 0;
    f.few = M <= kFp8StreamMaxM;
    f.rows = false;
    f.zeros = M > 0 && K == 0;
    if (f.zeros) std::memcpy(f.projs, projs, sizeof(wl_proj_fp8) * P);
    if (M == 0 || K == 0) return WL_OK;
    bool saved = x_codes != nullptr;  // a checkpoint is wanted
    Fp8RowsForward &sc = f.short_call;
    sc.nseg = 0;
    for (int i = 0; i < P; ++i) {
        const wl_proj_fp8 &q = projs[i];
        saved = saved || (q.T && q.r > 0);
        if (q.N > 0)
            sc.seg[sc.nseg++] = Fp8RowsSeg{q.codes, q.scales, q.s, bf16(q.U), bf16(q.V), bf16(q.y), q.N, q.r, 0};
    }
    sc.M = M;
    sc.K = K;
    sc.pitch = fp8_pitch(K);
    sc.x = bf16(x);
    if (!saved && plan_fp8_rows(sc)) {
        f.rows = true;
        return WL_OK;
    }
    uint8_t *codes = x_codes ? x_codes : l.codes, *scales = x_scales ? x_scales : l.scales;
    const Fp8Mat X{codes, scales, K, fp8_pitch(K)};
    int N[kMaxSeg], tiles = 0;  // tiles: counters of the few-token kernel
    for (int i = 0; i < P; ++i) {
        N[i] = projs[i].N;
        tiles += (N[i] + 127) / 128;
    }
    wl_status st;
    init_lowrank(f.lowrank, dev);
    __nv_bfloat16 *T[kMaxSeg];
    for (int i = 0; i < P; ++i) {
        const wl_proj_fp8 &q = projs[i];
        T[i] = q.T ? bf16(q.T) : l.T[i];
        if (q.r > 0 && (q.T || q.N > 0) &&
            (st = add_lowrank(f.lowrank, kLowrankRows, bf16(x), K, M, K, bf16(q.V), q.r, T[i], nullptr, f.lowrank.njobs > 0)) != WL_OK)
            return st;
    }
    plan_fp8_lowrank(f.lowrank, kLowrankRows, dev.sms);
    // One launch less where x is small: beside 2 M elements the few warps that
    // quantise there would be slower than a launch of their own.
    if (f.lowrank.njobs > 0 && (f.few || (long long)M * K <= 2 << 20)) {
        f.lowrank.quant = LowrankQuant{bf16(x), codes, scales, M, K, l.counters, f.few ? tiles : 0};
    } else {
        f.quant.job[0] = Fp8RowsJob{x, K, K, nullptr, codes, K, scales, nullptr, 0};
        f.quant.njobs = 1;
        f.quant.rows = M;
        f.quant.zero = l.counters;
        f.quant.n_zero = f.few ? tiles : 0;
    }
    // Weights fetched while the rank-r launch runs only take bandwidth from its read
    // of V (21504 -> 5376 at rank 256, 16 tokens: 34.2 us with the early fetch, 33.3
    // without; 128 tokens 56.5 and 55.5).
    const bool early = f.lowrank.njobs == 0;
    if (f.few) return set_stream(f.stream, X, M, K, projs, T, P, l.parts, l.counters, early, dev);
    Fp8GemmParams &g = f.gemm;
    init_gemm(g, M, N, P, (K + kFp8Block - 1) / kFp8Block, true, dev);
    for (int i = 0; i < P; ++i) {
        const wl_proj_fp8 &q = projs[i];
        if (q.N == 0) continue;
        const int k = g.nout;
        st = set_part(g, k, X, M, K, Fp8Mat{q.codes, q.scales, K, fp8_pitch(K)}, q.N, K, false, T[i], bf16(q.U), q.r, q.N, k > 0);
        if (st != WL_OK) return st;
        Fp8Out &o = add_out(g, q.N, k, 1);
        o.s = q.s;
        o.y = bf16(q.y);
    }
    return WL_OK;
}

wl_status forward_prepare(wl_fp8_plan &f, const wl_bf16 *x, int M, int K, const wl_proj_fp8 *projs, int P,
                          uint8_t *x_codes, uint8_t *x_scales, void *ws, size_t ws_bytes, Device &dev) {
    wl_status st = forward_check(x, M, K, projs, P, x_codes, x_scales);
    if (st != WL_OK) return st;
    const ForwardLayout l = forward_layout(M, K, projs, P, ws);
    if (M > 0 && K > 0 && (st = check_workspace(ws, ws_bytes, l.bytes)) != WL_OK) return st;
    if ((st = device_info(&dev.sms, &dev.status)) != WL_OK) return st;
    return forward_plan(f, x, M, K, projs, P, x_codes, x_scales, l, dev);
}

wl_status forward_launch(wl_fp8_plan &f, const Device &dev, cudaStream_t stream) {
    if (f.zeros) {
        for (int i = 0; i < f.P; ++i) {
            const wl_proj_fp8 &q = f.projs[i];
            if (q.N > 0 && cudaMemsetAsync(q.y, 0, (size_t)f.M * q.N * 2, stream) != cudaSuccess) return WL_ERR_CUDA;
            if (q.T && q.r > 0 && cudaMemsetAsync(q.T, 0, (size_t)f.M * q.r * 2, stream) != cudaSuccess)
                return WL_ERR_CUDA;
        }
        return WL_OK;
    }
    if (f.rows) return from_cuda(launch_fp8_rows(f.short_call, stream));
    if (f.quant.njobs > 0 && launch_fp8_quantize_rows(f.quant, WL_BF16, stream) != cudaSuccess) return WL_ERR_CUDA;
    if (launch_fp8_lowrank(f.lowrank, stream) != cudaSuccess) return WL_ERR_CUDA;
    return from_cuda(f.few ? launch_fp8_stream(f.stream, stream) : launch_fp8_gemm(f.gemm, kFp8Plain, dev.sms, stream));
}

// --------------------------------------------------------------- backward ----
struct BackwardLayout {
    uint8_t *g_codes[kMaxSeg], *g_scales[kMaxSeg];
    __nv_bfloat16 *E[kMaxSeg], *E_low[kMaxSeg];
    __nv_bfloat16 *dy[kMaxSeg];  // copies of gradients whose rows are not 16-byte aligned
    float *sums[kMaxSeg];
    size_t bytes;
};

// Ranges of the contraction in which ds is summed.
int sum_ranges(int K) { return std::max(1, (K + kFp8Block * kFp8RangeBlocks - 1) / (kFp8Block * kFp8RangeBlocks)); }

// Sizes alone: a copy of dy is laid out wherever one could be needed.
BackwardLayout backward_layout(int M, int K, const wl_grad_fp8 *projs, int P, void *ws) {
    BackwardLayout l = {};
    Arena a(ws);
    for (int i = 0; i < P; ++i) {
        l.g_codes[i] = a.take<uint8_t>((size_t)M * round16(projs[i].N));
        l.g_scales[i] = a.take<uint8_t>((size_t)M * fp8_pitch(projs[i].N));
        l.E[i] = a.take<__nv_bfloat16>((size_t)M * projs[i].r);
        l.E_low[i] = a.take<__nv_bfloat16>((size_t)M * projs[i].r);
        l.dy[i] = a.take<__nv_bfloat16>(projs[i].r > 0 ? (size_t)M * round16(projs[i].N) : 0);
        l.sums[i] = a.take<float>((size_t)sum_ranges(K) * ((M + 31) / 32) * projs[i].N);
    }
    l.bytes = a.used;
    return l;
}

wl_status backward_check(const uint8_t *x_codes, const uint8_t *x_scales, int M, int K, const wl_grad_fp8 *projs,
                         int P, const wl_bf16 *dx) {
    wl_status st = check_sizes(M, K, projs, P);
    const bool sizes_aligned = st != WL_ERR_ALIGNMENT;
    if (st != WL_OK && sizes_aligned) return st;
    if (M > 0 && K > 0 && (!x_codes || !x_scales)) return WL_ERR_INVALID_ARG;
    for (int i = 0; i < P; ++i) {
        const wl_grad_fp8 &q = projs[i];
        if (M == 0 || q.N == 0) continue;
        if (!q.dy || !q.s || (K > 0 && (!q.codes || !q.scales))) return WL_ERR_INVALID_ARG;
        if (q.r > 0 && (!q.U || !q.T || (K > 0 && !q.V))) return WL_ERR_INVALID_ARG;
    }
    if (!sizes_aligned) return WL_ERR_ALIGNMENT;
    if (!aligned(x_codes, 16) || !aligned(x_scales, 4) || !aligned(dx, 16)) return WL_ERR_ALIGNMENT;
    for (int i = 0; i < P; ++i) {
        const wl_grad_fp8 &q = projs[i];
        if (!aligned(q.codes, 16) || !aligned(q.scales, 4) || !aligned(q.s, 4) || !aligned(q.U, 16) ||
            !aligned(q.V, 16) || !aligned(q.T, 16) || !aligned(q.dy, 2) || !aligned(q.ds, 4) ||
            !aligned(q.dU, 16) || !aligned(q.dV, 16))
            return WL_ERR_ALIGNMENT;
    }
    return WL_OK;
}

// Gradients that are sums over nothing.
wl_status backward_zeros(int M, int K, const wl_grad_fp8 *projs, int P, wl_bf16 *dx, cudaStream_t stream) {
    for (int i = 0; i < P; ++i) {
        const wl_grad_fp8 &q = projs[i];
        if (q.ds && q.N > 0 && (M == 0 || K == 0) &&
            cudaMemsetAsync(q.ds, 0, (size_t)q.N * 4, stream) != cudaSuccess)
            return WL_ERR_CUDA;
        if (q.dU && q.N > 0 && q.r > 0 && M == 0 &&
            cudaMemsetAsync(q.dU, 0, (size_t)q.N * q.r * 2, stream) != cudaSuccess)
            return WL_ERR_CUDA;
        if (q.dV && K > 0 && q.r > 0 && (M == 0 || q.N == 0) &&
            cudaMemsetAsync(q.dV, 0, (size_t)K * q.r * 2, stream) != cudaSuccess)
            return WL_ERR_CUDA;
    }
    bool any = false;
    for (int i = 0; i < P; ++i) any = any || projs[i].N > 0;
    if (dx && !any && M > 0 && K > 0 && cudaMemsetAsync(dx, 0, (size_t)M * K * 2, stream) != cudaSuccess)
        return WL_ERR_CUDA;
    return WL_OK;
}

wl_status backward_run(const uint8_t *x_codes, const uint8_t *x_scales, int M, int K, const wl_grad_fp8 *projs, int P,
                       wl_bf16 *dx, const BackwardLayout &l, const Device &dev, cudaStream_t stream) {
    wl_status st = backward_zeros(M, K, projs, P, dx, stream);
    if (st != WL_OK || M == 0) return st;
    const Fp8Mat X{x_codes, x_scales, K, fp8_pitch(K)};
    Fp8GemmParams gx, gs;
    int N[kMaxSeg], blocks = 0;
    for (int i = 0; i < P; ++i) {
        N[i] = projs[i].N;
        blocks += (N[i] + kFp8Block - 1) / kFp8Block;
    }
    init_gemm(gx, M, &K, 1, blocks, true, dev);
    init_gemm(gs, M, N, P, (K + kFp8Block - 1) / kFp8Block, false, dev);
    Fp8RowsParams quant = {};
    quant.rows = M;
    Fp8SumParams sums = {};
    sums.n_rows = sum_ranges(K) * ((M + 31) / 32);
    LowrankParams le, lu, lv;
    init_lowrank(le, dev);
    init_lowrank(lu, dev);
    init_lowrank(lv, dev);
    int parts = 0;
    for (int i = 0; i < P; ++i) {
        const wl_grad_fp8 &q = projs[i];
        if (q.N == 0) continue;
        const Fp8Mat W{q.codes, q.scales, K, fp8_pitch(K)};
        const bool want_dv = q.dV && K > 0, want_dx = dx && K > 0;
        __nv_bfloat16 *copy = nullptr;
        if (q.r > 0 && (want_dv || want_dx || q.dU)) {
            const __nv_bfloat16 *dy = bf16(q.dy);
            long long ld = q.N;
            if (q.N % 8 != 0 || !aligned(q.dy, 16)) {  // copied, by the quantiser where it runs
                ld = round16(q.N);
                if (want_dx)
                    copy = l.dy[i];
                else if (launch_fp8_pad_rows(dy, M, q.N, l.dy[i], ld, stream) != cudaSuccess)
                    return WL_ERR_CUDA;
                dy = l.dy[i];
            }
            if ((want_dv || want_dx) && (st = add_lowrank(le, kLowrankRows, dy, ld, M, q.N, bf16(q.U), q.r, l.E[i],
                                                          want_dv ? l.E_low[i] : nullptr)) != WL_OK)
                return st;
            if (q.dU && (st = add_lowrank(lu, kLowrankCols, dy, ld, q.N, M, bf16(q.T), q.r, bf16(q.dU), nullptr)) != WL_OK)
                return st;
            if (want_dv && (st = add_lowrank_codes(lv, X, K, M, l.E[i], l.E_low[i], q.r, bf16(q.dV))) != WL_OK) return st;
        }
        if (q.ds && K > 0) {
            const int k = gs.nout;
            if ((st = set_part(gs, k, X, M, K, W, q.N, K, false, nullptr, nullptr, 0, 0, k > 0)) != WL_OK) return st;
            Fp8Out &o = add_out(gs, q.N, k, 1);
            o.dy = bf16(q.dy);
            o.sums = l.sums[i];
            sums.job[sums.njobs++] = Fp8SumJob{l.sums[i], q.ds, q.N, 0};
        }
        if (want_dx) {
            const long long ldg = round16(q.N);
            quant.job[quant.njobs++] = Fp8RowsJob{q.dy, q.N, q.N, q.s, l.g_codes[i], ldg, l.g_scales[i], copy, 0};
            if ((st = set_part(gx, parts, Fp8Mat{l.g_codes[i], l.g_scales[i], ldg, fp8_pitch(q.N)}, M, q.N, W, q.N, K, true,
                               l.E[i], bf16(q.V), q.r, K)) != WL_OK)
                return st;
            ++parts;
        }
    }
    plan_fp8_lowrank(le, kLowrankRows, dev.sms);
    plan_fp8_lowrank(lu, kLowrankCols, dev.sms);
    plan_fp8_lowrank(lv, kLowrankCodes, dev.sms);
    if (launch_fp8_quantize_rows(quant, WL_BF16, stream) != cudaSuccess ||
        launch_fp8_lowrank(le, stream) != cudaSuccess ||
        launch_fp8_lowrank(lu, stream) != cudaSuccess ||
        launch_fp8_lowrank(lv, stream) != cudaSuccess)
        return WL_ERR_CUDA;
    if (parts > 0) {
        Fp8Out &o = add_out(gx, K, 0, parts);
        o.y = bf16(dx);
        if (launch_fp8_gemm(gx, kFp8Transposed, dev.sms, stream) != cudaSuccess) return WL_ERR_CUDA;
    }
    gs.ranges = sum_ranges(K);
    gs.num_tiles *= gs.ranges;
    if (launch_fp8_gemm(gs, kFp8ColSums, dev.sms, stream) != cudaSuccess) return WL_ERR_CUDA;
    return from_cuda(launch_fp8_sum_rows(sums, stream));
}

}  // namespace
}  // namespace wl

extern "C" {

wl_status wl_quantize_fp8(const void *a, wl_type type, int rows, int cols, int block_rows, uint8_t *codes,
                          uint8_t *scales, void *stream_ptr) {
    using namespace wl;
    if (type != WL_BF16 && type != WL_F32) return WL_ERR_INVALID_ARG;
    if (block_rows != 1 && block_rows != kFp8Block) return WL_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0) return WL_ERR_INVALID_ARG;
    if (rows > kMaxSize || cols > kMaxSize) return WL_ERR_UNSUPPORTED;
    if (rows > 0 && cols > 0 && (!a || !codes || !scales)) return WL_ERR_INVALID_ARG;
    if (cols % 16 != 0 || !aligned(a, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return WL_ERR_ALIGNMENT;
    if (rows == 0 || cols == 0) return WL_OK;
    int sms, *status;
    wl_status st = device_info(&sms, &status);
    if (st != WL_OK) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (block_rows == kFp8Block) return from_cuda(launch_fp8_quantize_tiles(a, type, rows, cols, codes, scales, stream));
    Fp8RowsParams p = {};
    p.job[0] = Fp8RowsJob{a, cols, cols, nullptr, codes, cols, scales, nullptr, 0};
    p.njobs = 1;
    p.rows = rows;
    return from_cuda(launch_fp8_quantize_rows(p, type, stream));
}

}  // extern "C"

namespace wl {
namespace {

struct MatmulLayout {
    float *parts;
    unsigned int *counters;
    int tiles;  // counters to clear: 0 when no tile is cut
    size_t bytes;
};

MatmulLayout matmul_layout(int M, int N, int K, void *ws) {
    MatmulLayout l = {};
    Arena a(ws);
    if (M > 0 && M <= kFp8StreamMaxM && N > 0 && K > 0) {
        const int r = 0;
        Fp8StreamParams sp;
        plan_stream(sp, M, K, &N, &r, 1);
        l.tiles = sp.whole == sp.tiles ? 0 : sp.tiles;
        l.parts = a.take<float>(fp8_stream_part_floats(sp));
        l.counters = a.take<unsigned int>(l.tiles);
    }
    l.bytes = a.used;
    return l;
}

}  // namespace
}  // namespace wl

extern "C" {

size_t wl_matmul_fp8_workspace(int M, int N, int K) {
    using namespace wl;
    if (M > kMaxSize || N > kMaxSize || K > kMaxSize || K % 16 != 0) return 0;  // refused
    return matmul_layout(M, N, K, nullptr).bytes;
}

wl_status wl_matmul_fp8(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                        const uint8_t *b_scales, wl_bf16 *y, int M, int N, int K, void *workspace,
                        size_t workspace_bytes, void *stream_ptr) {
    using namespace wl;
    if (M < 0 || N < 0 || K < 0) return WL_ERR_INVALID_ARG;
    if (M > kMaxSize || N > kMaxSize || K > kMaxSize) return WL_ERR_UNSUPPORTED;
    if (M > 0 && N > 0) {
        if (!y) return WL_ERR_INVALID_ARG;
        if (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return WL_ERR_INVALID_ARG;
    }
    if (K % 16 != 0 || !aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 4) ||
        !aligned(b_scales, 4) || !aligned(y, 2))
        return WL_ERR_ALIGNMENT;
    if (M == 0 || N == 0) return WL_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (K == 0) return from_cuda(cudaMemsetAsync(y, 0, (size_t)M * N * 2, stream));
    const MatmulLayout l = matmul_layout(M, N, K, workspace);
    wl_status st = check_workspace(workspace, workspace_bytes, l.bytes);
    if (st != WL_OK) return st;
    Device dev;
    if ((st = device_info(&dev.sms, &dev.status)) != WL_OK) return st;
    if (M <= kFp8StreamMaxM) {
        if (l.tiles > 0 && cudaMemsetAsync(l.counters, 0, (size_t)l.tiles * sizeof(unsigned), stream) != cudaSuccess)
            return WL_ERR_CUDA;
        wl_proj_fp8 q = {};
        q.codes = b_codes;
        q.scales = b_scales;
        q.y = y;
        q.N = N;
        __nv_bfloat16 *T = nullptr;
        Fp8StreamParams sp;
        st = set_stream(sp, Fp8Mat{a_codes, a_scales, K, fp8_pitch(K)}, M, K, &q, &T, 1, l.parts, l.counters, false, dev);
        // y may be the weights of a bf16 call, which reads those before its wait
        sp.early_next = false;
        return st != WL_OK ? st : from_cuda(launch_fp8_stream(sp, stream));
    }
    Fp8GemmParams g;
    init_gemm(g, M, &N, 1, (K + kFp8Block - 1) / kFp8Block, true, dev);
    g.early_next = false;
    if ((st = set_part(g, 0, Fp8Mat{a_codes, a_scales, K, fp8_pitch(K)}, M, K, Fp8Mat{b_codes, b_scales, K, fp8_pitch(K)},
                       N, K, false, nullptr, nullptr, 0, 0)) != WL_OK)
        return st;
    add_out(g, N, 0, 1).y = bf16(y);
    return from_cuda(launch_fp8_gemm(g, kFp8Plain, dev.sms, stream));
}

size_t wl_stacked_forward_fp8_workspace(int M, int K, const wl_proj_fp8 *projs, int P) {
    using namespace wl;
    if (check_sizes(M, K, projs, P) != WL_OK) return 0;
    return forward_layout(M, K, projs, P, nullptr).bytes;
}

wl_status wl_stacked_forward_fp8(const wl_bf16 *x, int M, int K, const wl_proj_fp8 *projs, int P, uint8_t *x_codes,
                                 uint8_t *x_scales, void *workspace, size_t workspace_bytes, void *stream_ptr) {
    wl_fp8_plan f;
    wl::Device dev;
    wl_status st = wl::forward_prepare(f, x, M, K, projs, P, x_codes, x_scales, workspace, workspace_bytes, dev);
    return st != WL_OK ? st : wl::forward_launch(f, dev, static_cast<cudaStream_t>(stream_ptr));
}

wl_status wl_plan_stacked_forward_fp8(const wl_bf16 *x, int M, int K, const wl_proj_fp8 *projs, int P,
                                      uint8_t *x_codes, uint8_t *x_scales, void *workspace, size_t workspace_bytes,
                                      wl_fp8_plan **plan) {
    if (!plan) return WL_ERR_INVALID_ARG;
    *plan = nullptr;
    std::unique_ptr<wl_fp8_plan> f(new (std::nothrow) wl_fp8_plan);
    if (!f) return WL_ERR_NOMEM;
    wl::Device dev;
    wl_status st = wl::forward_prepare(*f, x, M, K, projs, P, x_codes, x_scales, workspace, workspace_bytes, dev);
    if (st == WL_OK) *plan = f.release();
    return st;
}

wl_status wl_run_fp8_plan(wl_fp8_plan *plan, void *stream) {
    if (!plan) return WL_ERR_INVALID_ARG;
    wl::Device dev;
    wl_status st = wl::device_info(&dev.sms, &dev.status);
    if (st != WL_OK) return st;
    plan->lowrank.timeout_ns = plan->stream.timeout_ns = plan->gemm.timeout_ns = wl::wait_limit_ns();
    return wl::forward_launch(*plan, dev, static_cast<cudaStream_t>(stream));
}

void wl_free_fp8_plan(wl_fp8_plan *plan) { delete plan; }

size_t wl_stacked_backward_fp8_workspace(int M, int K, const wl_grad_fp8 *projs, int P) {
    using namespace wl;
    if (check_sizes(M, K, projs, P) != WL_OK) return 0;
    return backward_layout(M, K, projs, P, nullptr).bytes;
}

wl_status wl_stacked_backward_fp8(const uint8_t *x_codes, const uint8_t *x_scales, int M, int K,
                                  const wl_grad_fp8 *projs, int P, wl_bf16 *dx, void *workspace,
                                  size_t workspace_bytes, void *stream_ptr) {
    using namespace wl;
    wl_status st = backward_check(x_codes, x_scales, M, K, projs, P, dx);
    if (st != WL_OK) return st;
    const BackwardLayout l = backward_layout(M, K, projs, P, workspace);
    if (M > 0 && (st = check_workspace(workspace, workspace_bytes, l.bytes)) != WL_OK) return st;
    Device dev;
    if ((st = device_info(&dev.sms, &dev.status)) != WL_OK) return st;
    return backward_run(x_codes, x_scales, M, K, projs, P, dx, l, dev, static_cast<cudaStream_t>(stream_ptr));
}

}  // extern "C"
