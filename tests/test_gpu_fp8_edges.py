"""GPU tests of 8-bit calls at the edges of what their kernels' plans cover."""
import ctypes
import threading

import pytest
import torch

import linear_wl_forward_b200 as wl
from oracle import fp8
from test_gpu_fp8 import bundle, cuda, done, f64, gen, host, tokens, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,r", [
    (1, 256, [256, 128], [1024, 0]), (16, 144, [300, 40], [0, 1024]), (128, 256, [256, 128], [648, 0]),
    (33, 16, [130, 1, 64], [8, 1024, 0]), (64, 256, [128, 128], [0, 1000])])
def test_short_projection_beside_a_long_one(M, K, N, r):
    """A projection of one unit (K <= 256, no delta) in a cluster whose size
    comes from a projection of many."""
    g = gen(M + K)
    x = tokens(g, M, K)
    projs = [bundle(g, n, K, q) for n, q in zip(N, r)]
    ys = wl.stacked_forward_fp8(x.cuda(), [cuda(p) for p in projs])
    done()
    for p, y in zip(projs, ys):
        within(y, fp8.forward(f64(x), *host(p))[0], "y")


def test_short_calls_from_two_host_threads():
    """Two host threads issue short calls of one kernel that need different
    amounts of shared memory."""
    g = gen(3)
    cases = []
    for K in (1152, 2048):
        x, dev = tokens(g, 8, K).cuda(), [cuda(bundle(g, 256, K, 0))]
        cases.append((x, dev, wl.stacked_forward_fp8(x, dev)[0].clone(), torch.cuda.Stream()))
    done()
    failed, start = [], threading.Barrier(len(cases))

    def run(x, dev, want, stream):
        try:
            handle, ys = wl.prepare_stacked_fp8(x, dev), None
            start.wait()
            for _ in range(4000):
                ys = handle(stream=stream)
            stream.synchronize()
            assert torch.equal(ys[0], want)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=run, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    done()
    assert not failed, failed


@pytest.mark.parametrize("M,K,N,r", [(16, 4112, [600], [64]), (3, 1040, [20000], [8]), (200, 528, [449, 30], [40, 8])])
def test_handle_dropped_while_its_call_runs(M, K, N, r):
    """The handle's memory, made on one stream and used on another, is not
    given out again before the call that uses it has ended."""
    g = gen(M)
    x, dev = tokens(g, M, K).cuda(), [cuda(bundle(g, n, K, q)) for n, q in zip(N, r)]
    want = wl.stacked_forward_fp8(x, dev)
    ys = [torch.empty_like(y) for y in want]
    done()
    for raw in (False, True):
        side = torch.cuda.Stream()
        handle = wl.prepare_stacked_fp8(x, dev, ys=ys)
        size = handle._ws.numel()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        handle(stream=side.cuda_stream if raw else side)
        del handle
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        done()
        assert all(torch.equal(a, b) for a, b in zip(ys, want)), (raw, len(junk))
        for y in ys:
            y.zero_()


def test_handle_refuses_a_stream_of_another_device():
    class Elsewhere:
        cuda_stream, device = 12345, torch.device("cuda", 7)

    g = gen(0)
    handle = wl.prepare_stacked_fp8(tokens(g, 3, 64).cuda(), [cuda(bundle(g, 40, 64, 8))])
    with pytest.raises(ValueError):
        handle(stream=Elsewhere())


@pytest.mark.parametrize("M,N,K", [(1024, 1152, 4096), (100, 5376, 2048), (128, 21504, 1152), (4096, 1152, 1152)])
def test_product_is_the_next_calls_weight(M, N, K):
    """y = A B^T as W0 of a bf16 call that directly follows: that call reads
    its weights ahead of its wait for the previous kernel."""
    g = gen(M)
    a = tuple(torch.from_numpy(t).cuda() for t in fp8.quantize(f64(tokens(g, M, K)), 1))
    codes, scales, *_ = bundle(g, N, K, 0)
    b = (codes.cuda(), scales.cuda())
    x, s = tokens(g, 1, N).cuda(), torch.ones(M, device="cuda")
    W = wl.matmul_fp8(a, b)
    done()
    want = wl.linear_forward(x, W, s, None, None)
    y = torch.empty_like(want)
    for _ in range(10):
        W.zero_()
        y.zero_()
        done()
        wl.matmul_fp8(a, b, y=W)
        wl.linear_forward(x, W, s, None, None, y=y)
        done()
        assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 3, 8, 40, 200])
@pytest.mark.parametrize("up", [60, -100, 118, -118, 119])
def test_scales_that_cancel(M, up):
    """Large weights with small tokens and the other way round: each product
    is of ordinary size, whatever its two scales are."""
    N, K = 200, 640
    g = gen(M + up)
    sign = torch.tensor([1.0, -1.0, 1.0, -1.0, 1.0]).repeat_interleave(128)
    x = (torch.randn(M, K, generator=g) * torch.exp2(-up * sign)).bfloat16()
    w = torch.randn(N, K, generator=g).double() * torch.exp2(up * sign.double())
    codes, scales = fp8.quantize(w.numpy(), 128)
    p = (torch.from_numpy(codes), torch.from_numpy(scales), torch.ones(N), None, None)
    y, = wl.stacked_forward_fp8(x.cuda(), [cuda(p)])
    done()
    within(y, fp8.forward(f64(x), *host(p))[0], "y")


def test_none_where_a_tensor_is_needed():
    g = gen(0)
    x, (codes, scales, s, U, V) = tokens(g, 4, 64).cuda(), cuda(bundle(g, 40, 64, 8))
    for call in (lambda: wl.stacked_forward_fp8(x, [(codes, scales, None, U, V)]),
                 lambda: wl.stacked_forward_fp8(x, [(codes, None, s, U, V)]),
                 lambda: wl.matmul_fp8(wl.quantize_fp8(x), (codes, None)),
                 lambda: wl.stacked_backward_fp8(wl.Fp8Checkpoint(*wl.quantize_fp8(x), [None]), [x[:, :40].contiguous()],
                                                 [(codes, scales, s, U, V)])):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("M,K,N,r", [(3, 1152, [1024, 256], [16, 0]), (16, 4112, [600], [64]), (200, 528, [449, 30], [40, 8])])
def test_plan_with_a_checkpoint(M, K, N, r):
    """The C plan that also leaves the checkpoint, run twice, against the call."""
    g = gen(M)
    dev = [cuda(bundle(g, n, K, q)) for n, q in zip(N, r)]
    x = tokens(g, M, K).cuda()
    L, u8, bf16 = wl.lib(), torch.uint8, torch.bfloat16
    ys = [torch.empty(M, n, dtype=bf16, device="cuda") for n in N]
    T = [torch.empty(M, q, dtype=bf16, device="cuda") if q else None for q in r]
    codes, scales = torch.empty(M, K, dtype=u8, device="cuda"), torch.empty(M, wl.fp8_scale_pitch(K), dtype=u8, device="cuda")
    xp, _, _, arr = wl._forward_fp8_args(x, dev, ys, T)
    n = L.wl_stacked_forward_fp8_workspace(M, K, arr, len(dev))
    ws, plan = torch.empty(n, dtype=u8, device="cuda"), ctypes.c_void_p()
    assert L.wl_plan_stacked_forward_fp8(xp, M, K, arr, len(dev), codes.data_ptr(), scales.data_ptr(), ws.data_ptr(), n,
                                         ctypes.byref(plan)) == 0
    try:
        for _ in range(2):
            x.copy_(tokens(g, M, K))
            ws.fill_(255)
            assert L.wl_run_fp8_plan(plan, torch.cuda.current_stream().cuda_stream) == 0
            want, ckpt = wl.stacked_forward_fp8(x, dev, checkpoint=True)
            done()
            assert all(torch.equal(a, b) for a, b in zip(ys, want))
            assert torch.equal(codes, ckpt.codes) and torch.equal(scales, ckpt.scales)
            assert all(a is b is None or torch.equal(a, b) for a, b in zip(T, ckpt.T))
    finally:
        L.wl_free_fp8_plan(plan)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_raw_handle_of_the_default_stream(M):
    """stream=0 is the default stream: behind what runs there already, and
    ahead of what comes after."""
    K, N, r = 1040, 300, 16
    g = gen(M)
    dev, x = [cuda(bundle(g, N, K, r))], tokens(g, M, K).cuda()
    dy = (1e-3 * torch.randn(M, N, generator=g)).bfloat16().cuda()
    want, ckpt = wl.stacked_forward_fp8(x, dev, checkpoint=True)
    plain = wl.stacked_forward_fp8(x, dev)
    wdx, wper = wl.stacked_backward_fp8(ckpt, [dy], dev)
    handle = wl.prepare_stacked_fp8(torch.zeros_like(x), dev)
    late = handle._keep[0]
    done()
    assert torch.cuda.current_stream().cuda_stream == 0
    torch.cuda._sleep(20_000_000)
    late.copy_(x)
    codes, scales = wl.quantize_fp8(late, stream=0)
    ys, saved = wl.stacked_forward_fp8(late, dev, checkpoint=True, stream=0)
    dx, per = wl.stacked_backward_fp8(saved, [dy], dev, stream=0)
    got = handle(stream=0)
    copies = [t.clone() for t in (codes, scales, ys[0], dx, *per[0], got[0])]
    done()
    for a, b in zip(copies, (ckpt.codes, ckpt.scales, want[0], wdx, *wper[0], plain[0])):
        assert torch.equal(a, b)
