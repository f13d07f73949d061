"""GPU tests of the 8-bit operators against the fp64 oracle.

Codes and scales must be equal.  Products are held element by element to the
bounds that oracle.fp8 derives: half a bf16 step of the result, half a bf16
step of each operand that is rounded, and two fp32 unit roundoffs per term of
a sum."""
import numpy as np
import pytest
import torch

import linear_wl_forward_b200 as wl
from oracle import fp8

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def done():
    torch.cuda.synchronize()
    assert wl.last_device_status() == 0


def within(got, want, what):
    value, bound = want
    got = f64(got)
    assert got.shape == value.shape, what
    d = np.abs(got - value)
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(d[bad] / np.maximum(bound[bad], 1e-300)):.3g} x bound at {np.argwhere(bad)[0]}"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def tokens(g, M, K):
    x = torch.randn(M, K, generator=g)
    x[:, torch.rand(K, generator=g) < 0.02] *= 20
    return x.bfloat16()


def bundle(g, N, K, r):
    codes, scales = fp8.quantize(0.02 * torch.randn(N, K, generator=g).double().numpy(), 128)
    s = 0.9 + 0.2 * torch.rand(N, generator=g)
    U = (0.02 * torch.randn(N, r, generator=g)).bfloat16() if r else None
    V = (0.02 * torch.randn(K, r, generator=g)).bfloat16() if r else None
    return torch.from_numpy(codes), torch.from_numpy(scales), s, U, V


def cuda(p):
    return tuple(None if t is None else t.cuda() for t in p)


def host(p):
    codes, scales, s, U, V = p
    return codes.numpy(), scales.numpy(), f64(s), None if U is None else f64(U), None if V is None else f64(V)


# --------------------------------------------------------------- quantiser ----
@pytest.mark.parametrize("rows,cols,block,dtype", [
    (1, 16, 1, torch.bfloat16), (3, 1152, 1, torch.bfloat16), (130, 528, 1, torch.float32), (17, 2064, 1, torch.bfloat16),
    (1, 16, 128, torch.bfloat16), (128, 128, 128, torch.float32), (129, 144, 128, torch.bfloat16),
    (300, 1040, 128, torch.float32), (5, 5376, 128, torch.bfloat16)])
def test_quantize(rows, cols, block, dtype):
    a = (torch.randn(rows, cols, generator=gen(rows + cols)) * torch.exp(3 * torch.randn(rows, 1, generator=gen(5)))).to(dtype)
    codes, scales = wl.quantize_fp8(a.cuda(), block_rows=block)
    done()
    want = fp8.quantize(f64(a), block)
    np.testing.assert_array_equal(scales.cpu().numpy(), want[1])
    np.testing.assert_array_equal(codes.cpu().numpy(), want[0])


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_special_values(block):
    a = torch.zeros(140, 400)
    a[0, :128] = 448.0 * 2.0 ** torch.arange(-64, 64)  # every binade against the largest
    a[0, 127] = float("inf")
    a[1, 5] = float("nan")
    a[2, 128:256] = float("-inf")  # a block without a finite element
    a[3, 256:384] = 1e-38  # smaller than the smallest scale's codes
    a[3, 300] = 1e-44
    a[4, 3] = 3.4e38
    a[129, 130] = 448.0
    a[130, 390] = float(np.nextafter(np.float32(448.0), np.float32(1e9)))  # one step over: the next scale
    a[131, 0] = -0.0
    codes, scales = wl.quantize_fp8(a.cuda(), block_rows=block)
    done()
    want = fp8.quantize(f64(a), block)
    np.testing.assert_array_equal(scales.cpu().numpy(), want[1])
    np.testing.assert_array_equal(codes.cpu().numpy(), want[0])


def test_quantize_ties():
    """Every midpoint of the E4M3 grid, on a row whose scale is 1."""
    grid = fp8.e4m3_decode(np.arange(127))
    row = np.zeros((1, 256), np.float32)
    row[0, :126] = (grid[:-1] + grid[1:]) / 2
    row[0, 127] = 448
    row[0, 128:254] = -row[0, :126]
    row[0, 255] = -448
    codes, scales = wl.quantize_fp8(torch.from_numpy(row).cuda())
    done()
    assert scales.cpu()[0, :2].tolist() == [127, 127]
    np.testing.assert_array_equal(codes.cpu().numpy(), fp8.e4m3_encode(row))


# ----------------------------------------------------------------- product ----
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 130, 128), (7, 300, 144), (16, 128, 1152), (48, 1024, 1152), (64, 257, 2064), (128, 225, 528),
    (129, 224, 512), (200, 449, 640), (257, 7, 4112), (300, 1000, 1040)])
def test_matmul(M, N, K):
    g = gen(M + N + K)
    a = fp8.quantize(f64(tokens(g, M, K)), 1)
    codes, scales, *_ = bundle(g, N, K, 0)
    y = wl.matmul_fp8(tuple(torch.from_numpy(t).cuda() for t in a), (codes.cuda(), scales.cuda()))
    done()
    within(y, fp8.matmul(a, (codes.numpy(), scales.numpy())), "y")


@pytest.mark.parametrize("M", [3, 150])
def test_matmul_scales_far_apart(M):
    """Block scales from 2^-40 to 2^40: each product takes its own."""
    N, K = 260, 1280
    g = gen(M)
    a = fp8.quantize(f64(tokens(g, M, K).float() * torch.exp2(torch.randint(-40, 41, (M, 1), generator=g).float())), 1)
    w = 0.02 * torch.randn(N, K, generator=g)
    w *= torch.exp2(torch.randint(-40, 41, (1, K // 128), generator=g).float()).repeat_interleave(128, 1)
    b = fp8.quantize(f64(w), 128)
    y = wl.matmul_fp8(tuple(torch.from_numpy(t).cuda() for t in a), tuple(torch.from_numpy(t).cuda() for t in b))
    done()
    within(y, fp8.matmul(a, b), "y")


def test_matmul_nan_stays_in_its_row():
    M, N, K = 140, 300, 256
    g = gen(9)
    x = f64(tokens(g, M, K))
    x[5, 200] = np.nan
    a = fp8.quantize(x, 1)
    codes, scales, *_ = bundle(g, N, K, 0)
    y = f64(wl.matmul_fp8(tuple(torch.from_numpy(t).cuda() for t in a), (codes.cuda(), scales.cuda())))
    done()
    assert np.isnan(y[5]).all() and np.isfinite(np.delete(y, 5, 0)).all()


# ----------------------------------------------------------------- forward ----
FORWARD = [
    # short calls: every token count, ranks up to 32, one to four row blocks per CTA
    (1, 1152, [1024, 256, 256], [16, 16, 16]), (2, 1152, [4096, 4096], [16, 8]), (3, 2048, [70, 3], [32, 0]),
    (4, 16, [200], [24]), (5, 352, [2500], [32]), (8, 400, [9000, 17], [8, 24]), (7, 2032, [16], [0]), (1, 2048, [500], [32]),
    (9, 1152, [1024], [16]), (1, 2064, [256], [16]), (1, 1152, [256], [40]),
    (1, 16, [1], [0]), (1, 128, [128], [8]), (1, 1152, [1024, 256, 256], [16, 16, 16]), (2, 5376, [300], [256]),
    (3, 272, [17, 0, 129], [8, 16, 0]), (5, 2064, [257], [72]), (8, 1024, [1152], [64]), (16, 1040, [1000, 8], [128, 256]),
    (17, 528, [130], [40]), (33, 144, [449], [8]), (64, 1152, [512, 512], [64, 64]), (100, 640, [225], [16]),
    (128, 512, [224], [0]), (129, 528, [300, 77], [16, 8]), (256, 256, [448], [64]), (333, 2000, [1001, 264, 77], [40, 0, 8]),
    (600, 384, [700], [320]), (40, 256, [64], [512]), (1, 256, [96], [1024]),
    # few tokens: whole tiles for every CTA, and tiles cut between them
    (2, 272, [19500, 300], [8, 16]), (20, 144, [40000], [0]), (1, 4112, [130], [0]), (128, 1040, [20000], [136]),
    # tiles cut along the contraction
    (200, 8208, [300], [72]), (513, 4112, [600, 31], [8, 0]), (140, 21504, [64], [256]),
    # tiles of 224 and of 128 columns, a second tile per CTA pair
    (2560, 272, [1568], [72]), (2560, 400, [890], [8]), (2816, 1296, [1121, 1000], [136, 0])]


@pytest.mark.parametrize("M,K,N,r", FORWARD)
def test_forward(M, K, N, r):
    g = gen(M * 7 + K)
    x = tokens(g, M, K)
    projs = [bundle(g, n, K, q) for n, q in zip(N, r)]
    dev = [cuda(p) for p in projs]
    ys, ckpt = wl.stacked_forward_fp8(x.cuda(), dev, checkpoint=True)
    plain = wl.stacked_forward_fp8(x.cuda(), dev)
    done()
    want = fp8.quantize(f64(x), 1)
    np.testing.assert_array_equal(ckpt.codes.cpu().numpy(), want[0])
    np.testing.assert_array_equal(ckpt.scales.cpu().numpy(), want[1])
    for p, y, y2, T in zip(projs, ys, plain, ckpt.T):
        wy, wT = fp8.forward(f64(x), *host(p))
        within(y, wy, "y")
        within(y2, wy, "y")  # a short call without a checkpoint has a kernel of its own
        if wT is not None:
            within(T, wT, "T")
        else:
            assert T is None


# ---------------------------------------------------------------- backward ----
@pytest.mark.parametrize("M,K,N,r", [
    (1, 16, [1], [8]), (1, 128, [128], [0]), (2, 1152, [1024, 256, 256], [16, 16, 16]), (5, 272, [17, 0, 129], [8, 16, 0]),
    (64, 1152, [512, 512], [64, 64]), (127, 528, [130], [40]), (200, 144, [449], [72]), (257, 640, [225, 31], [256, 8]),
    (333, 2000, [301, 264, 77], [40, 0, 8]), (512, 384, [700], [320]), (130, 256, [96], [1024]),
    # ds summed in ranges of the contraction
    (70, 20000, [300], [8]), (300, 8208, [130, 500], [0, 16]),
    # dx cut along the contraction
    (150, 304, [4000, 130], [8, 0]), (513, 272, [700, 900, 1300], [16, 0, 72]), (40, 64, [9000], [256]),
    # tiles of 224 and of 128 columns, a second tile per CTA pair
    (2560, 1568, [300, 77], [72, 0]), (2560, 896, [140], [16]), (2560, 272, [1568], [16]), (2816, 2128, [400, 1121], [136, 8])])
def test_backward(M, K, N, r):
    g = gen(M * 11 + K)
    x = tokens(g, M, K)
    projs = [bundle(g, n, K, q) for n, q in zip(N, r)]
    dys = [(1e-3 * torch.randn(M, n, generator=g)).bfloat16() for n in N]
    xc, xs = fp8.quantize(f64(x), 1)
    Ts = [None if p[3] is None else torch.from_numpy(f64(x) @ f64(p[4])).bfloat16() for p in projs]
    ckpt = wl.Fp8Checkpoint(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), [None if T is None else T.cuda() for T in Ts])
    dx, per = wl.stacked_backward_fp8(ckpt, [d.cuda() for d in dys], [cuda(p) for p in projs])
    done()
    wdx, wper = fp8.backward(xc, xs, [f64(d) for d in dys], [None if T is None else f64(T) for T in Ts], [host(p) for p in projs])
    within(dx, wdx, "dx")
    for (ds, dU, dV), (wds, wdU, wdV) in zip(per, wper):
        within(ds, wds, "ds")
        if wdU is None:
            assert dU is None and dV is None
        else:
            within(dU, wdU, "dU")
            within(dV, wdV, "dV")
