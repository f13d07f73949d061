"""CPU tests of the 8-bit oracle's norm bounds: a 128-column block left out of
a long contraction is far outside them, and correct rounding inside."""
import numpy as np
import pytest
import torch

from oracle import fp8
from test_gpu_fp8 import bundle, f64, gen, host, tokens


def bf16(a):
    return torch.from_numpy(np.asarray(a)).bfloat16().double().numpy()


@pytest.mark.parametrize("M,K,N,r", [(140, 21504, 64, 256), (70, 20000, 100, 8), (20, 8208, 130, 0)])
def test_norms_see_a_missing_block(M, K, N, r):
    g = gen(M)
    x, p = f64(tokens(g, M, K)), host(bundle(g, N, K, r))
    codes, scales, s, U, V = p
    y, tol = fp8.forward_norm(x, *p)
    rounded = fp8.dequantize(*fp8.quantize(x, 1), 1) @ fp8.dequantize(codes, scales, 128).T * s
    if r:
        rounded += bf16(x @ V) @ U.T
    assert fp8.norm(bf16(rounded) - y) <= tol
    gone = codes.copy()
    gone[:, -K % 128 + K - 256:-K % 128 + K - 128] = 0
    assert fp8.norm(fp8.forward_norm(x, gone, scales, s, U, V)[0] - y) > 2 * tol
    xc, xs = fp8.quantize(x, 1)
    dy = f64((1e-3 * torch.randn(M, N, generator=g)).bfloat16())
    ds, tol = fp8.ds_norm(xc, xs, dy, codes, scales, 8192)
    assert fp8.norm(ds.astype(np.float32) - ds) <= tol
    assert fp8.norm(fp8.ds_norm(xc, xs, dy, gone, scales, 8192)[0] - ds) > 2 * tol
    if r:
        v, tol = fp8.dv_norm(xc, xs, dy, U)
        assert fp8.norm(bf16(v) - v) <= tol


def test_norms_see_a_missing_block_of_rows():
    """dx, whose contraction runs over the projections' rows."""
    g = gen(1)
    M, K, N = 40, 64, [9000, 12000]
    projs = [host(bundle(g, n, K, 16)) for n in N]
    dys = [f64((1e-3 * torch.randn(M, n, generator=g)).bfloat16()) for n in N]
    dx, tol = fp8.dx_norm(dys, projs)
    assert fp8.norm(bf16(dx) - dx) <= tol
    codes, *rest = projs[1]
    gone = codes.copy()
    gone[1280:1408] = 0
    assert fp8.norm(fp8.dx_norm(dys, [projs[0], (gone, *rest)])[0] - dx) > 2 * tol
