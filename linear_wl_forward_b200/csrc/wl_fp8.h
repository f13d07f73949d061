// Parameter blocks and launchers of the 8-bit operators (E4M3 codes, E8M0
// scales per 128 columns), behind the C ABI in wl_fp8_api.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "wl_internal.h"

namespace wl {

constexpr int kFp8Block = 128;  // columns (and, for weights, rows) per scale

inline int fp8_pitch(int cols) { return WL_FP8_SCALE_PITCH(cols); }

// An fp8 matrix on the device.  ld: bytes from one row of codes to the next.
struct Fp8Mat {
    const uint8_t *codes;
    const uint8_t *scales;
    long long ld;
    int pitch;  // bytes per row of scales
};

// ----------------------------------------------------------- quantisation ----
// 1 x 128 blocks of rows of `a` (bf16 or fp32, `lda` elements apart), each
// element times colscale[column] first (nullptr: 1, bf16 only).  Rows of codes are ld_codes
// bytes apart, a multiple of 16; columns from `cols` up to ld_codes get code 0.
cudaError_t launch_fp8_quantize_rows(const void *a, wl_type type, long long lda, int rows, int cols,
                                     const float *colscale, uint8_t *codes, long long ld_codes,
                                     uint8_t *scales, cudaStream_t stream);
// 128 x 128 blocks; cols % 16 == 0, rows of codes cols bytes apart.
cudaError_t launch_fp8_quantize_tiles(const void *a, wl_type type, int rows, int cols, uint8_t *codes,
                                      uint8_t *scales, cudaStream_t stream);

// ---------------------------------------------------------------- products ----
// T[m][j] = sum_c X[m][c] V[c][j], bf16 out (X rows ldx elements apart).
cudaError_t launch_fp8_lowrank(const __nv_bfloat16 *X, long long ldx, int M, int C, const __nv_bfloat16 *V,
                               int r, __nv_bfloat16 *T, cudaStream_t stream);

// y = s (.) (A B^T) + T U^T; s nullptr: 1; r == 0: no second term.
cudaError_t launch_fp8_forward(const Fp8Mat &A, const Fp8Mat &B, int M, int N, int K, const float *s,
                               const __nv_bfloat16 *T, const __nv_bfloat16 *U, int r, __nv_bfloat16 *y,
                               cudaStream_t stream);

// acc (+)= G W + E V^T (fp32, M x K); out (bf16) written when not null.
cudaError_t launch_fp8_dgrad(const Fp8Mat &G, const Fp8Mat &W, int M, int N, int K, const __nv_bfloat16 *E,
                             const __nv_bfloat16 *V, int r, float *acc, bool add, __nv_bfloat16 *out,
                             cudaStream_t stream);

// ds[n] = sum_m dy[m][n] (A B^T)[m][n].
cudaError_t launch_fp8_ds(const Fp8Mat &A, const Fp8Mat &B, int M, int N, int K, const __nv_bfloat16 *dy,
                          float *ds, cudaStream_t stream);

// out[c][j] = sum_m X[m][c] B[m][j] for X in bf16 (dU), or in 8 bits (dV).
cudaError_t launch_fp8_tn_bf16(const __nv_bfloat16 *X, const __nv_bfloat16 *B, int M, int C, int r,
                               __nv_bfloat16 *out, cudaStream_t stream);
cudaError_t launch_fp8_tn_codes(const Fp8Mat &X, const __nv_bfloat16 *B, int M, int C, int r, __nv_bfloat16 *out,
                                cudaStream_t stream);

}  // namespace wl
