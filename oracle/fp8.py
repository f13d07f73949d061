"""fp64 oracle of the 8-bit operators (numpy): the block quantiser, the
block-scaled product, the theta-bundle forward with 8-bit W0 and activations,
and its backward from the 8-bit checkpoint.  Shares nothing with the CUDA
library.

An 8-bit matrix is E4M3 codes and a scale 2^E per block of block_rows x 128
elements; E is the smallest integer with 448 * 2^E >= max|a| over the block's
finite elements, at least -127, and 0 for a block of zeros.
"""
from __future__ import annotations

import numpy as np

# bf16 and fp32 half steps, relative to the value
U16, U32 = 2.0 ** -8, 2.0 ** -24


def scale_pitch(cols: int) -> int:
    return 4 * -(-cols // 512)


def e4m3_decode(codes):
    """Values of E4M3 bytes: sign, exponent (bias 7), mantissa; S.1111.111 is NaN."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


_GRID = e4m3_decode(np.arange(127))  # 0 .. 448, ascending


def e4m3_encode(v):
    """Nearest E4M3 byte (ties to the even code) of |v| <= 448; NaN and infinities give 0x7F."""
    v = np.asarray(v, np.float64)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.clip(np.searchsorted(_GRID, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code + np.where(np.signbit(v), 128, 0)
    return np.where(np.isfinite(v), code, 0x7F).astype(np.uint8)


def quantize(a, block_rows: int):
    """(codes R x C, scales) of a matrix."""
    a = np.asarray(a, np.float64)
    R, C = a.shape
    codes = np.zeros((R, C), np.uint8)
    scales = np.full((-(-R // block_rows), scale_pitch(C)), 127, np.uint8)
    for i in range(0, R, block_rows):
        for j in range(0, C, 128):
            b = a[i:i + block_rows, j:j + 128]
            top = np.max(np.abs(b[np.isfinite(b)]), initial=0.0)
            E = 0
            if top > 0:
                E = int(np.floor(np.log2(top))) - 10
                while 448.0 * 2.0 ** E < top:
                    E += 1
                E = max(E, -127)
            codes[i:i + block_rows, j:j + 128] = e4m3_encode(b / 2.0 ** E)
            scales[i // block_rows, j // 128] = E + 127
    return codes, scales


def dequantize(codes, scales, block_rows: int):
    R, C = codes.shape
    E = scales.astype(np.float64) - 127
    return e4m3_decode(codes) * np.exp2(E)[np.arange(R) // block_rows][:, np.arange(C) // 128]


def matmul(a, b):
    """(A B^T, bound on the error of a bf16 result summed in fp32)."""
    A, B = dequantize(*a, 1), dequantize(*b, 128)
    y = A @ B.T
    n = A.shape[1] + 8
    return y, U16 * np.abs(y) + 2 * n * U32 * (np.abs(A) @ np.abs(B).T)


def lowrank(X, V):
    """(X V, bound for fp32 sums rounded to bf16)."""
    X, V = np.asarray(X, np.float64), np.asarray(V, np.float64)
    T = X @ V
    return T, U16 * np.abs(T) + 2 * (X.shape[1] + 8) * U32 * (np.abs(X) @ np.abs(V))


def forward(x, codes, scales, s, U, V):
    """((y, bound), (T, bound)) of one projection.  The bound of y counts: its
    rounding to bf16, T's error carried through U, and one fp32 unit roundoff
    (doubled: the tensor cores may truncate) per term of each sum."""
    x = np.asarray(x, np.float64)
    X, W = dequantize(*quantize(x, 1), 1), dequantize(codes, scales, 128)
    s = np.asarray(s, np.float64)
    y = s * (X @ W.T)
    mag = np.abs(s) * (np.abs(X) @ np.abs(W).T)
    terms, err, T = x.shape[1] + 8, 0.0, None
    if U is not None:
        U = np.asarray(U, np.float64)
        T, eT = lowrank(x, V)
        y, mag = y + T @ U.T, mag + np.abs(T) @ np.abs(U).T
        err, terms, T = eT @ np.abs(U).T, terms + U.shape[1], (T, eT)
    err = err + 2 * terms * U32 * mag
    return (y, U16 * np.abs(y) + (1 + U16) * err), T


def backward(x_codes, x_scales, dys, Ts, projs):
    """dx and per projection ds, dU, dV, each as (value, bound)."""
    X = dequantize(x_codes, x_scales, 1)
    M = X.shape[0]
    dx, mag, err, terms, per = np.zeros_like(X), np.zeros_like(X), np.zeros_like(X), 8, []
    for (codes, scales, s, U, V), dy, T in zip(projs, dys, Ts):
        W = dequantize(codes, scales, 128)
        dy = np.asarray(dy, np.float64)
        # s (.) dy is formed in fp32 before it is quantised
        g = (np.asarray(s, np.float32) * dy.astype(np.float32)).astype(np.float64)
        G = dequantize(*quantize(g, 1), 1) if g.size else g
        dx, mag, terms = dx + G @ W, mag + np.abs(G) @ np.abs(W), terms + dy.shape[1]
        z, zmag = X @ W.T, np.abs(X) @ np.abs(W).T
        ds = ((dy * z).sum(0), 2 * (X.shape[1] + M + 8) * U32 * (np.abs(dy) * zmag).sum(0))
        dU = dV = None
        if U is not None:
            U, V, T = (np.asarray(a, np.float64) for a in (U, V, T))
            E, eE = lowrank(dy, U)
            dx, mag, err = dx + E @ V.T, mag + np.abs(E) @ np.abs(V).T, err + eE @ np.abs(V).T
            terms += U.shape[1]
            v = dy.T @ T
            dU = (v, U16 * np.abs(v) + 2 * (M + 8) * U32 * (np.abs(dy).T @ np.abs(T)))
            v, vmag = X.T @ E, np.abs(X).T @ np.abs(E)
            dV = (v, U16 * np.abs(v) + (1 + U16) * (np.abs(X).T @ eE + 2 * (M + 8) * U32 * vmag))
        per.append((ds, dU, dV))
    return (dx, U16 * np.abs(dx) + (1 + U16) * (err + 2 * terms * U32 * mag)), per


# ------------------------------------------------------------------- norms ----
# The bounds above grow with the number of terms and end as large as the values
# themselves (K = 20000).  These hold the Frobenius norm of an output's error,
# and see a single 128-column block that is left out of a long contraction.
#   * half a bf16 step of each element of the output: U16 of its norm;
#   * a bf16 operand's rounding E -> E + e, |e| <= U16 |E|, carried through B:
#     ||e B||_F <= U16 ||E||_F ||B||_2;
#   * fp32 sums on the tensor cores: a step adds 32 (8 bits) or 16 (bf16) terms
#     and is off by at most 2^-23 of the partial sum, whose norm over the matrix
#     stays below twice the result's: 2^-22 of it per step.
STEP = 2.0 ** -22


def norm(a):
    return float(np.linalg.norm(a))


def forward_norm(x, codes, scales, s, U, V):
    """(y, bound on the norm of its error) of one projection."""
    x = np.asarray(x, np.float64)
    X, W = dequantize(*quantize(x, 1), 1), dequantize(codes, scales, 128)
    y = np.asarray(s, np.float64) * (X @ W.T)
    tol = STEP * (x.shape[1] / 32) * norm(y)
    if U is not None:
        T, U = x @ np.asarray(V, np.float64), np.asarray(U, np.float64)
        y = y + T @ U.T
        tol += (U16 + STEP * (x.shape[1] + U.shape[1]) / 16) * norm(T) * np.linalg.norm(U, 2)
    return y, U16 * norm(y) + (1 + U16) * tol


def ds_norm(x_codes, x_scales, dy, codes, scales, run):
    """(ds, bound on the norm of its error) with sums of at most `run` columns on
    the tensor cores: each z = x^ W^T is off by STEP per step of its runs, which
    dy carries (Cauchy-Schwarz over the tokens), and the fp32 sums over runs and
    tokens by one unit per term."""
    X, W = dequantize(x_codes, x_scales, 1), dequantize(codes, scales, 128)
    dy, z = np.asarray(dy, np.float64), X @ W.T
    c = STEP * (run / 32) + (dy.shape[0] + X.shape[1] / run + 2) * U32
    return (dy * z).sum(0), c * norm(np.linalg.norm(dy, axis=0) * np.linalg.norm(z, axis=0))


def dx_norm(dys, projs):
    """(dx, bound on the norm of its error)."""
    dx, tol = 0.0, 0.0
    for (codes, scales, s, U, V), dy in zip(projs, dys):
        W, dy = dequantize(codes, scales, 128), np.asarray(dy, np.float64)
        g = (np.asarray(s, np.float32) * dy.astype(np.float32)).astype(np.float64)
        d = dequantize(*quantize(g, 1), 1) @ W
        dx, tol = dx + d, tol + STEP * (dy.shape[1] / 32) * norm(d)
        if U is not None:
            U, V = np.asarray(U, np.float64), np.asarray(V, np.float64)
            E = dy @ U
            dx = dx + E @ V.T
            tol += (U16 + STEP * (dy.shape[1] + U.shape[1]) / 16) * norm(E) * np.linalg.norm(V, 2)
    return dx, U16 * norm(dx) + (1 + U16) * tol


def dv_norm(x_codes, x_scales, dy, U):
    """(dV, bound on the norm of its error): E takes part in two bf16 terms,
    which leave at most U16^2 of it."""
    X, dy, U = dequantize(x_codes, x_scales, 1), np.asarray(dy, np.float64), np.asarray(U, np.float64)
    E = dy @ U
    v = X.T @ E
    tol = (U16 * U16 + STEP * (dy.shape[1] + X.shape[0]) / 16) * np.linalg.norm(X, 2) * norm(E)
    return v, U16 * norm(v) + (1 + U16) * tol
