// C ABI of the 8-bit operators: argument checks, the workspace's layout and
// the order of the launches.  Contracts in include/wl.h.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

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
        T *p = reinterpret_cast<T *>(base + used);
        used += (n * sizeof(T) + 255) & ~size_t(255);
        return base ? p : nullptr;
    }
};

constexpr int kWsAlign = 16;

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
    for (int i = 0; i < P; ++i) {
        if (projs[i].N < 0 || projs[i].r < 0) return WL_ERR_INVALID_ARG;
        if (projs[i].r > WL_MAX_RANK) return WL_ERR_UNSUPPORTED;
    }
    if (K % 16 != 0) return WL_ERR_ALIGNMENT;
    for (int i = 0; i < P; ++i)
        if (projs[i].r % 8 != 0) return WL_ERR_ALIGNMENT;
    return WL_OK;
}

struct ForwardLayout {
    uint8_t *codes, *scales;
    __nv_bfloat16 *T[kMaxSeg];
    size_t bytes;
};

ForwardLayout forward_layout(int M, int K, const wl_proj_fp8 *projs, int P, void *ws) {
    ForwardLayout l = {};
    Arena a(ws);
    l.codes = a.take<uint8_t>((size_t)M * K);
    l.scales = a.take<uint8_t>((size_t)M * fp8_pitch(K));
    for (int i = 0; i < P; ++i) l.T[i] = a.take<__nv_bfloat16>((size_t)M * projs[i].r);
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

wl_status forward_run(const wl_bf16 *x_, int M, int K, const wl_proj_fp8 *projs, int P, uint8_t *x_codes,
                      uint8_t *x_scales, const ForwardLayout &l, cudaStream_t stream) {
    const __nv_bfloat16 *x = reinterpret_cast<const __nv_bfloat16 *>(x_);
    uint8_t *codes = x_codes ? x_codes : l.codes, *scales = x_scales ? x_scales : l.scales;
    cudaError_t e = launch_fp8_quantize_rows(x, WL_BF16, K, M, K, nullptr, codes, K, scales, stream);
    if (e != cudaSuccess) return WL_ERR_CUDA;
    const int pitch = fp8_pitch(K);
    for (int i = 0; i < P; ++i) {
        const wl_proj_fp8 &q = projs[i];
        __nv_bfloat16 *T = q.T ? reinterpret_cast<__nv_bfloat16 *>(q.T) : l.T[i];
        if (q.r > 0 && (q.T || q.N > 0)) {
            e = launch_fp8_lowrank(x, K, M, K, reinterpret_cast<const __nv_bfloat16 *>(q.V), q.r, T, stream);
            if (e != cudaSuccess) return WL_ERR_CUDA;
        }
        if (q.N == 0) continue;
        e = launch_fp8_forward(Fp8Mat{codes, scales, K, pitch}, Fp8Mat{q.codes, q.scales, K, pitch}, M, q.N, K, q.s, T,
                               reinterpret_cast<const __nv_bfloat16 *>(q.U), q.r,
                               reinterpret_cast<__nv_bfloat16 *>(q.y), stream);
        if (e != cudaSuccess) return WL_ERR_CUDA;
    }
    return WL_OK;
}

// --------------------------------------------------------------- backward ----
struct BackwardLayout {
    uint8_t *g_codes[kMaxSeg], *g_scales[kMaxSeg];
    __nv_bfloat16 *E[kMaxSeg];
    float *dx;
    size_t bytes;
};

BackwardLayout backward_layout(int M, int K, const wl_grad_fp8 *projs, int P, void *ws) {
    BackwardLayout l = {};
    Arena a(ws);
    l.dx = a.take<float>((size_t)M * K);
    for (int i = 0; i < P; ++i) {
        l.g_codes[i] = a.take<uint8_t>((size_t)M * round16(projs[i].N));
        l.g_scales[i] = a.take<uint8_t>((size_t)M * fp8_pitch(projs[i].N));
        l.E[i] = a.take<__nv_bfloat16>((size_t)M * projs[i].r);
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
                       wl_bf16 *dx, const BackwardLayout &l, cudaStream_t stream) {
    wl_status st = backward_zeros(M, K, projs, P, dx, stream);
    if (st != WL_OK || M == 0) return st;
    const Fp8Mat X{x_codes, x_scales, K, fp8_pitch(K)};
    bool add = false;
    int last = -1;
    for (int i = 0; i < P; ++i)
        if (projs[i].N > 0) last = i;
    for (int i = 0; i < P; ++i) {
        const wl_grad_fp8 &q = projs[i];
        if (q.N == 0) continue;
        const __nv_bfloat16 *dy = reinterpret_cast<const __nv_bfloat16 *>(q.dy);
        const __nv_bfloat16 *U = reinterpret_cast<const __nv_bfloat16 *>(q.U);
        const __nv_bfloat16 *V = reinterpret_cast<const __nv_bfloat16 *>(q.V);
        const Fp8Mat W{q.codes, q.scales, K, fp8_pitch(K)};
        cudaError_t e = cudaSuccess;
        if (q.r > 0) e = launch_fp8_lowrank(dy, q.N, M, q.N, U, q.r, l.E[i], stream);
        if (e == cudaSuccess && q.dU && q.r > 0)
            e = launch_fp8_tn_bf16(dy, reinterpret_cast<const __nv_bfloat16 *>(q.T), M, q.N, q.r,
                                   reinterpret_cast<__nv_bfloat16 *>(q.dU), stream);
        if (e == cudaSuccess && q.dV && q.r > 0 && K > 0)
            e = launch_fp8_tn_codes(X, l.E[i], M, K, q.r, reinterpret_cast<__nv_bfloat16 *>(q.dV), stream);
        if (e == cudaSuccess && q.ds && K > 0) e = launch_fp8_ds(X, W, M, q.N, K, dy, q.ds, stream);
        if (e == cudaSuccess && dx && K > 0) {
            const long long ldg = round16(q.N);
            e = launch_fp8_quantize_rows(dy, WL_BF16, q.N, M, q.N, q.s, l.g_codes[i], ldg, l.g_scales[i], stream);
            if (e == cudaSuccess)
                e = launch_fp8_dgrad(Fp8Mat{l.g_codes[i], l.g_scales[i], ldg, fp8_pitch(q.N)}, W, M, q.N, K, l.E[i], V,
                                     q.r, l.dx, add, i == last ? reinterpret_cast<__nv_bfloat16 *>(dx) : nullptr,
                                     stream);
            add = true;
        }
        if (e != cudaSuccess) return WL_ERR_CUDA;
    }
    return WL_OK;
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
    if (rows > 0 && cols > 0 && (!a || !codes || !scales)) return WL_ERR_INVALID_ARG;
    if (cols % 16 != 0 || !aligned(a, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return WL_ERR_ALIGNMENT;
    if (rows == 0 || cols == 0) return WL_OK;
    int sms, *status;
    wl_status st = device_info(&sms, &status);
    if (st != WL_OK) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    return from_cuda(block_rows == 1
                         ? launch_fp8_quantize_rows(a, type, cols, rows, cols, nullptr, codes, cols, scales, stream)
                         : launch_fp8_quantize_tiles(a, type, rows, cols, codes, scales, stream));
}

size_t wl_matmul_fp8_workspace(int M, int N, int K) {
    (void)M, (void)N, (void)K;
    return 0;
}

wl_status wl_matmul_fp8(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                        const uint8_t *b_scales, wl_bf16 *y, int M, int N, int K, void *workspace,
                        size_t workspace_bytes, void *stream_ptr) {
    using namespace wl;
    if (M < 0 || N < 0 || K < 0) return WL_ERR_INVALID_ARG;
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
    wl_status st = check_workspace(workspace, workspace_bytes, wl_matmul_fp8_workspace(M, N, K));
    if (st != WL_OK) return st;
    int sms, *status;
    if ((st = device_info(&sms, &status)) != WL_OK) return st;
    return from_cuda(launch_fp8_forward(Fp8Mat{a_codes, a_scales, K, fp8_pitch(K)},
                                        Fp8Mat{b_codes, b_scales, K, fp8_pitch(K)}, M, N, K, nullptr, nullptr, nullptr,
                                        0, reinterpret_cast<__nv_bfloat16 *>(y), stream));
}

size_t wl_stacked_forward_fp8_workspace(int M, int K, const wl_proj_fp8 *projs, int P) {
    using namespace wl;
    if (check_sizes(M, K, projs, P) != WL_OK) return 0;
    return forward_layout(M, K, projs, P, nullptr).bytes;
}

wl_status wl_stacked_forward_fp8(const wl_bf16 *x, int M, int K, const wl_proj_fp8 *projs, int P, uint8_t *x_codes,
                                 uint8_t *x_scales, void *workspace, size_t workspace_bytes, void *stream_ptr) {
    using namespace wl;
    wl_status st = forward_check(x, M, K, projs, P, x_codes, x_scales);
    if (st != WL_OK || M == 0) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (K == 0) {  // x W0^T = 0 and x V = 0
        for (int i = 0; i < P; ++i) {
            const wl_proj_fp8 &q = projs[i];
            if (q.N > 0 && cudaMemsetAsync(q.y, 0, (size_t)M * q.N * 2, stream) != cudaSuccess) return WL_ERR_CUDA;
            if (q.T && q.r > 0 && cudaMemsetAsync(q.T, 0, (size_t)M * q.r * 2, stream) != cudaSuccess)
                return WL_ERR_CUDA;
        }
        return WL_OK;
    }
    const ForwardLayout l = forward_layout(M, K, projs, P, workspace);
    if ((st = check_workspace(workspace, workspace_bytes, l.bytes)) != WL_OK) return st;
    int sms, *status;
    if ((st = device_info(&sms, &status)) != WL_OK) return st;
    return forward_run(x, M, K, projs, P, x_codes, x_scales, l, stream);
}

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
    int sms, *status;
    if ((st = device_info(&sms, &status)) != WL_OK) return st;
    return backward_run(x_codes, x_scales, M, K, projs, P, dx, l, static_cast<cudaStream_t>(stream_ptr));
}

}  // extern "C"
