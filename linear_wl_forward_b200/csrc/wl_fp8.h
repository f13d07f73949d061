// Parameter blocks and launchers of the 8-bit operators (E4M3 codes, E8M0
// scales per 128 columns), behind the C ABI in wl_fp8_api.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "wl_internal.h"

namespace wl {

constexpr int kFp8Block = 128;  // columns (and, for weights, rows) per scale
// The plans estimate a call's cycles.  An SM was measured to take 46 bytes per
// cycle into shared memory in the long GEMM; the rates in the estimates are the
// ones whose choices were fastest for each kernel, and hold its other costs too.
constexpr double kFp8GemmFill = 42, kFp8StreamFill = 42, kFp8LowrankFill = 48;

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
// element times colscale[column] first (nullptr: 1; bf16 only).  Rows of codes
// are ld_codes bytes apart, a multiple of 16; columns from `cols` up to
// ld_codes get code 0.
struct Fp8RowsJob {
    const void *a;
    long long lda;
    int cols;
    const float *colscale;
    uint8_t *codes;
    long long ld_codes;
    uint8_t *scales;
    __nv_bfloat16 *copy;   // with column scales: a copy of `a`, rows ld_codes elements apart, or nullptr
    long long warp_begin;  // filled by the launcher
};
// One matrix, or up to kMaxSeg bf16 ones with column scales, of `rows` rows in
// one launch, which also clears n_zero words at `zero`.
struct Fp8RowsParams {
    Fp8RowsJob job[kMaxSeg];
    int njobs, rows;
    unsigned int *zero;
    int n_zero;
};
cudaError_t launch_fp8_quantize_rows(Fp8RowsParams &p, wl_type type, cudaStream_t stream);
// 128 x 128 blocks; cols % 16 == 0, rows of codes cols bytes apart.
cudaError_t launch_fp8_quantize_tiles(const void *a, wl_type type, int rows, int cols, uint8_t *codes,
                                      uint8_t *scales, cudaStream_t stream);

// Rows of `a` copied to rows `ld` elements apart, zeros behind column `cols`.
cudaError_t launch_fp8_pad_rows(const __nv_bfloat16 *a, int rows, int cols, __nv_bfloat16 *out, long long ld,
                                cudaStream_t stream);

// ---------------------------------------------------- products of rank r ----
// out[i][j] = sum_k A(i, k) B[k][j] for up to kMaxSeg products in one launch.
enum LowrankMode {
    kLowrankRows = 0,  // A row-major in i, bf16
    kLowrankCols,      // A row-major in k, bf16
    kLowrankCodes,     // A row-major in k, 8 bits with 1 x 128 blocks along i; B in two bf16 terms
    kLowrankFew        // Rows with up to 16 rows: chosen by the plan
};

// Rows of A per tile that are loaded (Rows mode).
inline int lowrank_a_rows(int I) { return I >= 128 ? 128 : (I + 15) / 16 * 16; }

struct LowrankJob {
    CUtensorMap tm_a;   // box 64 columns x lowrank_a_rows rows (Rows), 64 x 64 (Cols), 32 words x 64 rows, not swizzled (Codes)
    CUtensorMap tm_b;   // K x r, box 64 x 64
    CUtensorMap tm_b2;  // Codes: the low term
    const uint8_t *a_scales;
    int a_pitch;
    int I, K, r;
    int kb;             // 64-row blocks of the contraction
    __nv_bfloat16 *out;      // I x r
    __nv_bfloat16 *out_low;  // what rounding `out` to bf16 left over, or nullptr
    int tile_begin;
};

// Rows mode, every job with this A: the launch also quantises A (rows x cols,
// bf16, dense) in 1 x 128 blocks and clears n_zero words; a == nullptr: nothing.
struct LowrankQuant {
    const __nv_bfloat16 *a;
    uint8_t *codes, *scales;
    int rows, cols;
    unsigned int *zero;
    int n_zero;
};

struct LowrankParams {
    LowrankJob job[kMaxSeg];
    int njobs;
    LowrankQuant quant;
    LowrankMode mode;  // plan, with the next line
    int BN, split, tiles, stages, a_bytes, stage_bytes, tmem_cols;
    int *status;
    unsigned long long timeout_ns;
};

void plan_fp8_lowrank(LowrankParams &p, LowrankMode mode, int num_sms);
cudaError_t launch_fp8_lowrank(const LowrankParams &p, cudaStream_t stream);

// -------------------------------------------------------------------- GEMM ----
// Tensor-core product over CTA pairs: output tiles of 256 rows x 224, 128 or 64 columns (BN),
//   out[m][n] = s[n] * sum over parts, k of A[m][k] B[n][k]  +  sum over parts, j of T[m][j] U[n][j]
// with A in 8 bits (1 x 128 blocks along the contraction) and B in 8 bits
// (128 x 128 blocks).  The forward has one output per projection, each with
// one part; dx has one output whose parts are the projections.
constexpr int kFp8BM = 256;      // rows per CTA pair, 128 per CTA
constexpr int kFp8GemmThreads = 384;
constexpr int kFp8Stages = 3;
constexpr int kFp8BlockBytes = 32768;  // 16 KB of A (or T), up to 16 KB of B (or U)
constexpr int kFp8StageBytes = 2 * kFp8BlockBytes;
constexpr int kFp8RangeBlocks = 64;  // blocks of the contraction per range of column sums
constexpr int kFp8SfSlots = 4;
constexpr int kFp8SfBytes = 1536;      // four blocks of scales: 128 rows of A, 256 of B

struct Fp8Part {
    const uint8_t *a_scales, *b_scales;
    int a_pitch, b_pitch;
    int nkb;  // blocks of the contraction
    int lr;   // 64-column blocks of T and U, 0 = none
};

struct Fp8Out {
    const float *s;        // nullptr: 1
    __nv_bfloat16 *y;      // rows N elements apart
    int N;
    int part0, nparts;
    int tile_begin;
    // column sums instead of y (kFp8ColSums)
    const __nv_bfloat16 *dy;  // M x N
    float *sums;              // [ranges][ceil(M / 32)][N]: sums over 32 rows of dy (.) (A B^T)
};

struct Fp8GemmParams {
    CUtensorMap tm_a[kMaxSeg];  // codes, box 128 bytes x 128 rows
    CUtensorMap tm_b[kMaxSeg];  // codes, box 128 bytes x BN / 2 rows; transposed: 128, 64 or 32 bytes x 128 rows
    CUtensorMap tm_t[kMaxSeg];  // bf16, box 64 x 128 rows
    CUtensorMap tm_u[kMaxSeg];  // bf16, box 64 x BN / 2 rows
    Fp8Part part[kMaxSeg];
    Fp8Out out[kMaxSeg];
    int nout;
    int M, BN;
    int split;        // CTA pairs that share a tile
    // Column sums: ranges of the contraction that a tile is summed in, one after
    // the other.  The tensor cores' sums are cut off, not rounded, at each step,
    // so their error grows with their length (2e-6 of ds at 20000 columns).
    int ranges;
    int m_tiles, num_tiles;
    int early_next;   // the next kernel may start at once; not where it may read `y` before its wait
    int *status;
    unsigned long long timeout_ns;
};

enum Fp8Mode {
    kFp8Plain = 0,    // B rows run over the output columns (K-major)
    kFp8Transposed,   // B rows run over the contraction (N-major): dx
    kFp8ColSums       // K-major, the epilogue forms column sums: ds
};

// Sets BN, split, ranges (1) and m_tiles for M rows (set), outputs of N[0..nout) columns and
// a contraction of `blocks` blocks.
void plan_fp8_gemm(Fp8GemmParams &p, const int *N, int nout, int blocks, bool may_split, int num_sms);
cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, Fp8Mode mode, int num_sms, cudaStream_t stream);
// ds[n] = sum over rows i < n_rows of sums[i][n], for several outputs in one launch.
struct Fp8SumJob {
    const float *sums;
    float *ds;
    int N, cta_begin;  // cta_begin: filled by the launcher
};
struct Fp8SumParams {
    Fp8SumJob job[kMaxSeg];
    int njobs, n_rows;
};
cudaError_t launch_fp8_sum_rows(Fp8SumParams &p, cudaStream_t stream);

// ------------------------------------------------------- few-token stream ----
constexpr int kFp8StreamMaxM = 128;
constexpr int kFp8StreamMaxCluster = 16;
constexpr int kFp8StreamMaxGrid = 148;  // CTAs, whatever the device: the cut is made before one is known, and no CTA waits for another

struct Fp8StreamSeg {
    const uint8_t *w_scales;
    const float *s;      // nullptr: 1
    __nv_bfloat16 *y;    // M x N
    int N;
    int nkb, lr;         // 128-column blocks of the contraction, 64-column blocks of U
    // plan
    int kpairs, units;   // pairs of the contraction's blocks; with those of U
    long long unit_begin;
    int tile_begin;
};

struct Fp8StreamParams {
    CUtensorMap tm_w[kMaxSeg];  // codes, box 128 bytes x 128 rows
    CUtensorMap tm_u[kMaxSeg];  // bf16, box 64 x 128 rows
    CUtensorMap tm_t[kMaxSeg];  // bf16, box 64 x Mp rows
    CUtensorMap tm_x;           // codes, box 128 bytes x Mp rows
    Fp8StreamSeg seg[kMaxSeg];
    const uint8_t *x_scales;
    int pitch;
    int nseg, M;
    int early;  // the weights may be read before the wait for the previous kernel
    int early_next;  // as in Fp8GemmParams
    // plan
    int Mp, stages, grid, tiles;
    int whole;               // tiles [0, whole) go to one CTA (or cluster) each
    int cluster;             // CTAs per whole tile; above 1 all tiles are whole
    int cut_ctas;            // CTAs that share the others
    long long units, cut_unit;  // units, and those of the whole tiles
    float *parts;            // [cut_ctas][2][Mp][128]
    unsigned int *counters;  // [tiles], zero
    int *status;
    unsigned long long timeout_ns;
};

// Needs nseg, M and each segment's N, nkb and lr.
void plan_fp8_stream(Fp8StreamParams &p);
size_t fp8_stream_part_floats(const Fp8StreamParams &p);
cudaError_t launch_fp8_stream(const Fp8StreamParams &p, cudaStream_t stream);

// -------------------------------------------------- short calls, one launch ----
constexpr int kFp8RowsMaxK = 2048;

struct Fp8RowsSeg {
    const uint8_t *codes, *w_scales;
    const float *s;
    const __nv_bfloat16 *U, *V;
    __nv_bfloat16 *y;  // M x N
    int N, r;
    int cta_begin;     // plan
};

struct Fp8RowsForward {
    Fp8RowsSeg seg[kMaxSeg];
    int nseg;
    int M, K, pitch;
    const __nv_bfloat16 *x;
    int blocks, grid;  // plan: 16-row blocks per CTA, CTAs
};

// False if the call is not short enough; needs everything but the plan.
bool plan_fp8_rows(Fp8RowsForward &p);
cudaError_t launch_fp8_rows(const Fp8RowsForward &p, cudaStream_t stream);

}  // namespace wl
