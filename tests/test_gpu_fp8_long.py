"""GPU tests of the 8-bit operators on long contractions and small terms, where
the element-wise bounds of the oracle are as large as the values: exact
integers, norms of the errors, and sums that a lost term shows in."""
import numpy as np
import pytest
import torch

import linear_wl_forward_b200 as wl
from oracle import fp8
from test_gpu_fp8 import bundle, cuda, done, f64, gen, host, tokens
from test_gpu_fp8_use import exact_case, small_ints

pytestmark = pytest.mark.gpu


def near(got, want, what):
    value, tol = want
    err = fp8.norm(f64(got) - value)
    assert err <= tol, f"{what}: {err:.3g}, bound {tol:.3g}, norm {fp8.norm(value):.3g}"


# (short and long calls, tiles cut along the contraction, ds in ranges)
LONG = [(140, 21504, [64], [256]), (16, 21504, [300], [64]), (1, 16400, [130, 20], [16, 0]), (70, 20000, [300], [8]),
        (300, 8208, [130, 500], [0, 16]), (33, 24592, [129], [40])]


@pytest.mark.parametrize("M,K,N,r", LONG)
def test_long_integers_exact(M, K, N, r):
    x, W, projs = exact_case(M, K, N, r, seed=K)
    dev = [cuda(p) for p in projs]
    ys, ckpt = wl.stacked_forward_fp8(x.cuda(), dev, checkpoint=True)
    plain = wl.stacked_forward_fp8(x.cuda(), dev)
    dys = [small_ints(gen(7), -1, 1, M, n).bfloat16() for n in N]
    dx, per = wl.stacked_backward_fp8(ckpt, [d.cuda() for d in dys], dev)
    done()
    X, want_dx = x.double(), torch.zeros(M, K, dtype=torch.float64)
    for (codes, scales, s, U, V), w, y, y2, T, dy, (ds, dU, dV) in zip(projs, W, ys, plain, ckpt.T, dys, per):
        w, s, d = w.double(), s.double(), dy.double()
        z = X @ w.T
        want = s * z
        want_dx += (d * s) @ w
        if U is not None:
            t, E = X @ V.double(), d @ U.double()
            want += t @ U.double().T
            want_dx += E @ V.double().T
            assert torch.equal(T.double().cpu(), t)
            assert torch.equal(dU.cpu(), (d.T @ t).bfloat16())
            assert torch.equal(dV.cpu(), (X.T @ E).bfloat16())
        assert torch.equal(y.cpu(), want.bfloat16()) and torch.equal(y2, y)
        assert torch.equal(ds.double().cpu(), (d * z).sum(0))
    assert torch.equal(dx.cpu(), want_dx.bfloat16())


@pytest.mark.parametrize("M,K,N,r", LONG + [(512, 1152, [9000], [16]), (40, 64, [9000, 12000], [16, 0])])
def test_norms(M, K, N, r):
    g = gen(M * 3 + K)
    x = tokens(g, M, K)
    projs = [bundle(g, n, K, q) for n, q in zip(N, r)]
    dys = [(1e-3 * torch.randn(M, n, generator=g)).bfloat16() for n in N]
    dev = [cuda(p) for p in projs]
    ys, ckpt = wl.stacked_forward_fp8(x.cuda(), dev, checkpoint=True)
    plain = wl.stacked_forward_fp8(x.cuda(), dev)
    dx, per = wl.stacked_backward_fp8(ckpt, [d.cuda() for d in dys], dev)
    done()
    xc, xs = ckpt.codes.cpu().numpy(), ckpt.scales.cpu().numpy()
    hosts, dy64 = [host(p) for p in projs], [f64(d) for d in dys]
    for p, y, y2, dy, (ds, dU, dV) in zip(hosts, ys, plain, dy64, per):
        want = fp8.forward_norm(f64(x), *p)
        near(y, want, "y")
        near(y2, want, "y without a checkpoint")
        near(ds, fp8.ds_norm(xc, xs, dy, p[0], p[1], 8192), "ds")
        if p[3] is not None:
            near(dV, fp8.dv_norm(xc, xs, dy, p[3]), "dV")
    near(dx, fp8.dx_norm(dy64, hosts), "dx")


@pytest.mark.parametrize("M", [1, 40, 300])
def test_ds_is_summed_in_ranges(M):
    """2^24, then 256 ones, one per 32 columns, then -2^24, each in a range of
    its own: a sum that meets the ones at 2^24 loses them."""
    K, N = 24576, 40
    x, W = torch.zeros(M, K), torch.zeros(N, K)
    x[:, 0], x[:, 16384] = 2.0 ** 12, 2.0 ** 12
    W[:, 0], W[:, 16384] = 2.0 ** 12, -2.0 ** 12
    x[:, 8192:16384:32] = 1
    W[:, 8192:16384:32] = 1
    codes, scales = fp8.quantize(W.double().numpy(), 128)
    dev = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.ones(N, device="cuda"), None, None)
    ckpt = wl.Fp8Checkpoint(*wl.quantize_fp8(x.bfloat16().cuda()), [None])
    _, [(ds, _, _)] = wl.stacked_backward_fp8(ckpt, [torch.ones(M, N, dtype=torch.bfloat16, device="cuda")], [dev], need_dx=False)
    done()
    assert (ds == 256.0 * M).all(), ds


@pytest.mark.parametrize("M,N", [(2, 300), (40, 600), (200, 300), (700, 5000)])
def test_dv_takes_e_in_two_terms(M, N):
    """E = 257 and -256 in two tokens with x = 1: dV = 1, and 0 if E were rounded to bf16."""
    K, r = 272, 8
    x, dy, U = torch.zeros(M, K), torch.zeros(M, N), torch.zeros(N, r)
    x[0], x[M - 1] = 1, 1
    dy[0, :257], dy[M - 1, :256] = 1, -1
    U[:, ::2] = 1
    g = gen(0)
    codes, scales, s, _, V = cuda(bundle(g, N, K, r))
    ckpt = wl.Fp8Checkpoint(*wl.quantize_fp8(x.bfloat16().cuda()), [torch.zeros(M, r, dtype=torch.bfloat16, device="cuda")])
    _, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dy.bfloat16().cuda()], [(codes, scales, s, U.bfloat16().cuda(), V)])
    done()
    assert (dV[:, ::2] == 1).all() and (dV[:, 1::2] == 0).all()


@pytest.mark.parametrize("M", [5, 60, 200])
def test_dv_of_the_smallest_scales(M):
    """Codes whose values lie below 2^-126 down to 2^-136: bf16 holds multiples
    of 2^-133, so an expanded code is off by at most 2^-134."""
    K, N, r = 272, 130, 8
    g = gen(M)
    codes = torch.randint(0, 256, (M, K), generator=g).to(torch.uint8)
    codes[(codes & 127) == 127] = 3
    scales = torch.full((M, 4), 127, dtype=torch.uint8)
    scales[:, :3] = torch.randint(0, 8, (M, 3), generator=g).to(torch.uint8)
    wc, wsc, s, U, V = bundle(g, N, K, r)
    U = (U.float() * 2.0 ** 60).bfloat16()
    dy = (torch.randn(M, N, generator=g) * 2.0 ** 60).bfloat16()
    ckpt = wl.Fp8Checkpoint(codes.cuda(), scales.cuda(), [torch.zeros(M, r, dtype=torch.bfloat16, device="cuda")])
    _, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dy.cuda()], [cuda((wc, wsc, s, U, V))], need_dx=False)
    done()
    value, tol = fp8.dv_norm(codes.numpy(), scales.numpy(), f64(dy), f64(U))
    E = f64(dy) @ f64(U)
    near(dV, (value, tol + 2.0 ** -134 * np.sqrt(M * K) * fp8.norm(E)), "dV")
    # where every value is at least 2^-127 no bits are lost
    big = scales.clone()
    big[:, :3] = 9
    ckpt = wl.Fp8Checkpoint(codes.cuda(), big.cuda(), ckpt.T)
    _, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dy.cuda()], [cuda((wc, wsc, s, U, V))], need_dx=False)
    done()
    near(dV, fp8.dv_norm(codes.numpy(), big.numpy(), f64(dy), f64(U)), "dV")
