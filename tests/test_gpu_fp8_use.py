"""GPU tests of how the 8-bit operators are used: together from the host
decomposition on, on exact values, on side streams, in captured graphs, at
once, with unaligned and empty inputs, and when a wait gives up."""
import numpy as np
import pytest
import torch

import linear_wl_forward_b200 as wl
from oracle import fp8
from test_gpu_fp8 import bundle, cuda, done, f64, gen, host, tokens, within

pytestmark = pytest.mark.gpu


def small_ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g).float()


def exact_case(M, K, N, r, seed=0):
    """Integers that every step holds exactly (|sums| stay below 256 in bf16 outputs' range of exactness)."""
    g = gen(seed)
    x = small_ints(g, -1, 1, M, K).bfloat16()
    W = [small_ints(g, -1, 1, n, K) * (torch.rand(n, K, generator=g) < 16 / K) for n in N]
    projs = []
    for n, q, w in zip(N, r, W):
        codes, scales = fp8.quantize(w.double().numpy(), 128)
        s = torch.exp2(small_ints(g, 0, 1, n))
        U = (small_ints(g, -1, 1, n, q) * (torch.rand(n, q, generator=g) < 4 / q)).bfloat16() if q else None
        V = (small_ints(g, -1, 1, K, q) * (torch.rand(K, q, generator=g) < 16 / K)).bfloat16() if q else None
        projs.append((torch.from_numpy(codes), torch.from_numpy(scales), s, U, V))
    return x, W, projs


@pytest.mark.parametrize("M,K,N,r", [(1, 1152, [1000, 40], [16, 0]), (33, 2064, [300], [72]), (200, 528, [257, 129], [8, 136]),
                                     (700, 4112, [500], [40])])
def test_integers_exact(M, K, N, r):
    x, W, projs = exact_case(M, K, N, r)
    dev = [cuda(p) for p in projs]
    ys, ckpt = wl.stacked_forward_fp8(x.cuda(), dev, checkpoint=True)
    dys = [small_ints(gen(7), -1, 1, M, n).bfloat16() for n in N]
    dx, per = wl.stacked_backward_fp8(ckpt, [d.cuda() for d in dys], dev)
    done()
    X = x.double()
    want_dx = torch.zeros(M, K, dtype=torch.float64)
    for (codes, scales, s, U, V), w, y, T, dy, (ds, dU, dV) in zip(projs, W, ys, ckpt.T, dys, per):
        w, s, d = w.double(), s.double(), dy.double()
        want, E = s * (X @ w.T), None
        want_dx += (d * s) @ w
        if U is not None:
            t, E = X @ V.double(), d @ U.double()
            want += t @ U.double().T
            want_dx += E @ V.double().T
            assert torch.equal(T.double().cpu(), t)
            # sums past 256 round to bf16 once
            assert torch.equal(dU.cpu(), (d.T @ t).bfloat16())
            assert torch.equal(dV.cpu(), (X.T @ E).bfloat16())
        assert torch.equal(y.cpu(), want.bfloat16())
        assert torch.equal(ds.double().cpu(), (d * (X @ w.T)).sum(0))
    assert torch.equal(dx.cpu(), want_dx.bfloat16())


@pytest.mark.parametrize("M", [1, 24, 300])
def test_gradients_against_differences(M):
    """f is linear in s, U and V at fixed codes: a step of one argument moves
    sum(dy * y) by its gradient, exactly on exact values."""
    x, W, projs = exact_case(M, 528, [140], [24], seed=3)
    (codes, scales, s, U, V) = cuda(projs[0])
    _, ckpt = wl.stacked_forward_fp8(x.cuda(), [(codes, scales, s, U, V)], checkpoint=True)
    dy = small_ints(gen(5), -1, 1, M, 140).bfloat16().cuda()
    dx, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dy], [(codes, scales, s, U, V)])

    def f(x=x.cuda(), s=s, U=U, V=V):
        return float((wl.stacked_forward_fp8(x, [(codes, scales, s, U, V)])[0].double() * dy.double()).sum())

    base = f()
    rng = np.random.default_rng(0)
    for name, arg, grad in (("s", s, ds), ("U", U, dU), ("V", V, dV), ("x", x.cuda(), dx)):
        for _ in range(5):
            at = tuple(int(rng.integers(0, d)) for d in arg.shape)
            if abs(float(grad[at])) > 256:
                continue  # rounded
            moved = arg.clone()
            moved[at] += 1
            assert f(**{name: moved}) - base == float(grad[at]), (name, at)
    done()


def test_from_the_decomposition_to_a_step():
    """The whole run: band mean from the host decomposition, its blocks put
    into 8 bits, forward with a checkpoint, backward, a step of s, U and V that
    lowers the squared error against the dense layer."""
    rng = np.random.default_rng(1)
    L_, N, K, r, M = 2, 160, 144, 8, 192
    dense = (0.05 * rng.standard_normal((1, N, K)) + 0.02 * rng.standard_normal((L_, N, K))).astype(np.float32)
    W0, s, U, V, _ = wl.decompose(dense, 1, r)
    codes, scales = wl.quantize_fp8(torch.from_numpy(W0[0]).cuda(), block_rows=128)
    want = fp8.quantize(W0[0].astype(np.float64), 128)
    np.testing.assert_array_equal(codes.cpu().numpy(), want[0])
    proj = (codes, scales, torch.from_numpy(s[0]).cuda(), torch.from_numpy(U[0]).bfloat16().cuda(), torch.from_numpy(V[0]).bfloat16().cuda())
    x = tokens(gen(2), M, K).cuda()
    target = x.double() @ torch.from_numpy(dense[0]).double().cuda().T
    (y,), ckpt = wl.stacked_forward_fp8(x, [proj], checkpoint=True)
    dy = ((y.double() - target) / M).bfloat16()
    dx, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dy], [proj])
    done()
    hp = host(tuple(t.cpu() for t in proj))
    wy, wT = fp8.forward(f64(x), *hp)
    within(y, wy, "y")
    within(ckpt.T[0], wT, "T")
    wdx, [(wds, wdU, wdV)] = fp8.backward(ckpt.codes.cpu().numpy(), ckpt.scales.cpu().numpy(), [f64(dy)], [f64(ckpt.T[0])], [hp])
    within(dx, wdx, "dx")
    within(ds, wds, "ds")
    within(dU, wdU, "dU")
    within(dV, wdV, "dV")
    assert all(torch.isfinite(t.float()).all() for t in (dx, ds, dU, dV))


@pytest.mark.parametrize("M", [2, 40, 300])
def test_follows_its_weights_kernel_and_side_streams(M):
    """The forward right behind the kernel that writes its weights, on a side
    stream that starts from them, without any synchronisation in between."""
    N, K, r = 300, 1040, 16
    g = gen(M)
    w = (0.02 * torch.randn(N, K, generator=g)).cuda()
    x = tokens(g, M, K).cuda()
    _, _, s, U, V = cuda(bundle(g, N, K, r))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for scale in (1.0, 2.0, 4.0):
        with torch.cuda.stream(side):
            codes, scales = wl.quantize_fp8(w * scale, 128)
            outs.append(wl.stacked_forward_fp8(x, [(codes, scales, s, U, V)])[0])
    codes, scales = wl.quantize_fp8(w, 128, stream=side)
    handle = wl.stacked_forward_fp8(x, [(codes, scales, s, U, V)], stream=side)[0]
    raw = wl.stacked_forward_fp8(x, [(codes, scales, s, U, V)], stream=side.cuda_stream)[0]
    side.synchronize()
    for scale, y in zip((1.0, 2.0, 4.0), outs):
        wy, _ = fp8.forward(f64(x), *fp8.quantize(f64(w * scale), 128), f64(s), f64(U), f64(V))
        within(y, wy, f"scale {scale}")
    assert torch.equal(handle, outs[0]) and torch.equal(raw, outs[0])


@pytest.mark.parametrize("M,K,N,r", [(1, 1152, [1024, 256], [16, 16]), (16, 5376, [300], [64]), (7, 272, [20000], [8]), (300, 528, [449], [40])])
def test_captured_and_replayed(M, K, N, r):
    """Two graphs of the same call and a prepared one, replayed in turn with
    other inputs, against eager calls; a backward captured while an eager one
    lives."""
    g = gen(M)
    dev = [cuda(bundle(g, n, K, q)) for n, q in zip(N, r)]
    xs = [tokens(g, M, K).cuda() for _ in range(3)]
    dys = [[(1e-3 * torch.randn(M, n, generator=g)).bfloat16().cuda() for n in N] for _ in range(3)]
    eager = []
    for x, dy in zip(xs, dys):
        ys, ckpt = wl.stacked_forward_fp8(x, dev, checkpoint=True)
        # (a short call without a checkpoint has a kernel of its own)
        eager.append((ys, ckpt, wl.stacked_backward_fp8(ckpt, dy, dev), wl.stacked_forward_fp8(x, dev)))
    x, dy = xs[0].clone(), [d.clone() for d in dys[0]]
    handle = wl.prepare_stacked_fp8(x, dev)
    handle()
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ys, ckpt = wl.stacked_forward_fp8(x, dev, checkpoint=True)
            dx, per = wl.stacked_backward_fp8(ckpt, dy, dev)
            hy = handle()
        graphs.append((gr, ys, ckpt, dx, per, hy))
    for i in (1, 2, 0):
        x.copy_(xs[i])
        for a, b in zip(dy, dys[i]):
            a.copy_(b)
        for gr, ys, ckpt, dx, per, hy in graphs:
            gr.replay()
            torch.cuda.synchronize()
            ey, eckpt, (edx, eper), eplain = eager[i]
            assert all(torch.equal(a, b) for a, b in zip(ys + hy, ey + eplain))
            assert torch.equal(ckpt.codes, eckpt.codes) and torch.equal(dx, edx)
            for p, q in zip(per, eper):
                assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(p, q))
    done()


def test_two_calls_at_once():
    """Different calls on two streams, many times: nothing is shared."""
    g = gen(1)
    cases = []
    for M, K, N, r in [(16, 4112, [600], [64]), (3, 1040, [20000], [8]), (200, 528, [449, 30], [40, 8]), (2560, 272, [1568], [16])]:
        x, dev = tokens(g, M, K).cuda(), [cuda(bundle(g, n, K, q)) for n, q in zip(N, r)]
        cases.append((x, dev, wl.stacked_forward_fp8(x, dev)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(12):
        for i, st in enumerate(streams):
            x, dev, want = cases[(rep + 2 * i + rep // 4) % 4]
            got.append((wl.stacked_forward_fp8(x, dev, stream=st), want))
    done()
    for ys, want in got:
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("M,N", [(3, 40), (5, 129), (150, 264), (300, 77)])
def test_unaligned_outputs_and_gradients(M, N, offset):
    """y and dy that start inside a buffer; nothing around y is written."""
    K, r = 272, 16
    g = gen(M + N)
    x, p = tokens(g, M, K), bundle(g, N, K, r)
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[offset:offset + M * N].view(M, N)
    wl.stacked_forward_fp8(x.cuda(), [cuda(p)], ys=[y])
    done()
    want, T = fp8.forward(f64(x), *host(p))
    within(y, want, "y")
    assert (buf[:offset] == 7).all() and (buf[offset + M * N:] == 7).all()
    dyb = (1e-3 * torch.randn(M * N + 64, generator=g)).bfloat16()
    dy = dyb[offset:offset + M * N].view(M, N)
    _, ckpt = wl.stacked_forward_fp8(x.cuda(), [cuda(p)], checkpoint=True)
    dev = dyb.cuda()[offset:offset + M * N].view(M, N)
    dx, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dev], [cuda(p)])
    done()
    wdx, [(wds, wdU, wdV)] = fp8.backward(ckpt.codes.cpu().numpy(), ckpt.scales.cpu().numpy(), [f64(dy)], [f64(ckpt.T[0])], [host(p)])
    for got, want, name in ((dx, wdx, "dx"), (ds, wds, "ds"), (dU, wdU, "dU"), (dV, wdV, "dV")):
        within(got, want, name)


def test_empty_sizes():
    g = gen(0)
    p = cuda(bundle(g, 40, 64, 8))
    ys, ckpt = wl.stacked_forward_fp8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), [p], checkpoint=True)
    assert ys[0].shape == (0, 40)
    dx, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [ys[0]], [p])
    done()
    assert dx.shape == (0, 64) and not ds.any() and not dU.any() and not dV.any()
    none = cuda(bundle(g, 0, 64, 8))
    x = tokens(g, 5, 64).cuda()
    (y0, y1), ckpt = wl.stacked_forward_fp8(x, [none, p], checkpoint=True)
    assert y0.shape == (5, 0) and torch.equal(y1, wl.stacked_forward_fp8(x, [p])[0])
    dx, per = wl.stacked_backward_fp8(ckpt, [y0, y1], [none, p])
    alone = wl.stacked_backward_fp8(wl.Fp8Checkpoint(ckpt.codes, ckpt.scales, ckpt.T[1:]), [y1], [p])
    done()
    assert torch.equal(dx, alone[0]) and not per[0][2].any() and torch.equal(per[1][1], alone[1][0][1])
    dx, per = wl.stacked_backward_fp8(wl.Fp8Checkpoint(ckpt.codes, ckpt.scales, ckpt.T[:1]), [y0], [none])
    done()
    assert not dx.any()
    # K = 0: products over nothing
    x = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    p = (torch.empty(9, 0, dtype=torch.uint8, device="cuda"), torch.empty(1, 0, dtype=torch.uint8, device="cuda"),
         torch.ones(9, device="cuda"), torch.ones(9, 8, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"))
    (y,), ckpt = wl.stacked_forward_fp8(x, [p], checkpoint=True)
    assert torch.equal(wl.prepare_stacked_fp8(x, [p])()[0], y)
    dy = torch.ones(3, 9, dtype=torch.bfloat16, device="cuda")
    dx, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [dy], [p])
    done()
    assert not y.any() and not ckpt.T[0].any() and not ds.any() and not dU.any() and dx.shape == (3, 0)
    assert wl.matmul_fp8((x.view(torch.uint8).view(3, 0), torch.empty(3, 0, dtype=torch.uint8, device="cuda")), p[:2]).abs().sum() == 0


@pytest.mark.parametrize("M", [4, 60, 300])
def test_nonfinite_and_dropped_gradients(M):
    K, N, r = 400, 260, 16
    g = gen(M)
    x, p = tokens(g, M, K), cuda(bundle(g, N, K, r))
    bad = x.clone()
    bad[1, 7], bad[2, 300] = float("nan"), float("inf")
    want = wl.stacked_forward_fp8(x.cuda(), [p])[0]
    y = wl.stacked_forward_fp8(bad.cuda(), [p])[0]
    done()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(y[keep], want[keep]) and torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    _, ckpt = wl.stacked_forward_fp8(x.cuda(), [p], checkpoint=True)
    dy = (1e-3 * torch.randn(M, N, generator=g)).bfloat16()
    full = wl.stacked_backward_fp8(ckpt, [dy.cuda()], [p])
    only_x = wl.stacked_backward_fp8(ckpt, [dy.cuda()], [p], need_params=False)
    only_p = wl.stacked_backward_fp8(ckpt, [dy.cuda()], [p], need_dx=False)
    badd = dy.clone()
    badd[3, 11] = float("nan")
    dx, [(ds, dU, dV)] = wl.stacked_backward_fp8(ckpt, [badd.cuda()], [p])
    done()
    assert torch.equal(full[0], only_x[0]) and only_x[1] == [(None, None, None)] and only_p[0] is None
    assert all(torch.equal(a, b) for a, b in zip(full[1][0], only_p[1][0]))
    keep = [i for i in range(M) if i != 3]
    assert torch.equal(dx[keep], full[0][keep]) and torch.isnan(dx[3]).all()
    others = [i for i in range(N) if i != 11]
    assert torch.isnan(ds[11]) and torch.equal(ds[others], full[1][0][0][others])
    assert torch.isnan(dU[11].float()).all() and torch.equal(dU[others], full[1][0][1][others])


def test_python_refusals():
    g = gen(0)
    x, p = tokens(g, 4, 64).cuda(), cuda(bundle(g, 40, 64, 8))
    with pytest.raises(TypeError):
        wl.stacked_forward_fp8(x.float(), [p])
    with pytest.raises(ValueError):
        wl.stacked_forward_fp8(x, [(p[0][:, :48], *p[1:])])
    with pytest.raises(ValueError):
        wl.stacked_forward_fp8(x, [(p[0].t().contiguous().t(), *p[1:])])
    with pytest.raises(ValueError):
        wl.stacked_forward_fp8(x, [(*p[:4], None)])
    with pytest.raises(ValueError):
        wl.stacked_forward_fp8(x, [p], ys=[])
    with pytest.raises(TypeError):
        wl.quantize_fp8(x.half())
    with pytest.raises(ValueError):
        wl.quantize_fp8(x, block_rows=32)
    with pytest.raises(wl.WLError):
        wl.quantize_fp8(torch.zeros(4, 40, device="cuda"))
    with pytest.raises(wl.WLError):
        wl.stacked_forward_fp8(x, [p] * 9)
    with pytest.raises(ValueError):
        wl.stacked_backward_fp8(wl.Fp8Checkpoint(*wl.quantize_fp8(x), [None]), [x, x], [p])


def test_results_repeat():
    g = gen(4)
    for M, K, N, r in [(5, 4112, [700], [64]), (16, 1040, [20000], [8]), (260, 4112, [300], [136])]:
        x, dev = tokens(g, M, K).cuda(), [cuda(bundle(g, n, K, q)) for n, q in zip(N, r)]
        dy = [(1e-3 * torch.randn(M, n, generator=g)).bfloat16().cuda() for n in N]
        runs = []
        for _ in range(3):
            ys, ckpt = wl.stacked_forward_fp8(x, dev, checkpoint=True)
            dx, per = wl.stacked_backward_fp8(ckpt, dy, dev)
            runs.append(ys + ckpt.T + [dx] + [t for q in per for t in q])
        done()
        assert all(torch.equal(a, b) for q in runs[1:] for a, b in zip(runs[0], q))


@pytest.mark.parametrize("M,K,N,r", [(8, 4112, [600], [64]), (4, 1040, [20000], [8]), (300, 2064, [449], [40]), (300, 4112, [64], [8])])
def test_a_wait_that_gives_up(M, K, N, r):
    """With a wait limit of 1 ns a call either records the time-out or is
    right (one try of a wait may itself last until the data are there); the
    next call with the default limit is right either way."""
    g = gen(M)
    x, dev = tokens(g, M, K).cuda(), [cuda(bundle(g, n, K, q)) for n, q in zip(N, r)]
    want, ckpt = wl.stacked_forward_fp8(x, dev, checkpoint=True)
    grads = wl.stacked_backward_fp8(ckpt, want, dev)
    done()
    wl.set_wait_limit(1)
    try:
        for _ in range(10):
            ys = wl.stacked_forward_fp8(x, dev)
            status = wl.STATUS[wl.last_device_status()]
            assert status == "WL_ERR_TIMEOUT" or status == "WL_OK" and torch.equal(ys[0], want[0])
            dx, _ = wl.stacked_backward_fp8(ckpt, want, dev)
            status = wl.STATUS[wl.last_device_status()]
            assert status == "WL_ERR_TIMEOUT" or status == "WL_OK" and torch.equal(dx, grads[0])
    finally:
        wl.set_wait_limit(0)
    again = wl.stacked_forward_fp8(x, dev)
    dx, _ = wl.stacked_backward_fp8(ckpt, want, dev)
    done()
    assert torch.equal(again[0], want[0]) and torch.equal(dx, grads[0])
