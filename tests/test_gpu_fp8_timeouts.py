"""The 8-bit kernels' bounded waits, made to give up: with a wait limit of 1 ns
calls whose waits are long (contractions of 20000 columns and more) record
WL_ERR_TIMEOUT, a call that does not is right, and the next call with the
default limit is right again.  Every wait is bounded, and the kernels let
their copies and MMAs in flight end before their CTAs exit."""
import ctypes

import pytest
import torch

import linear_wl_forward_b200 as wl
from test_gpu_fp8 import done

pytestmark = pytest.mark.gpu

TIMEOUT = 5


def must_expire(call, tries=10):
    """`call` returns a list of tensors; at least one of the tries gives up."""
    want = [t.clone() for t in call()]
    done()
    wl.set_wait_limit(1)
    seen = []
    try:
        for _ in range(tries):
            got = call()
            seen.append(wl.last_device_status())
            assert seen[-1] in (0, TIMEOUT)
            assert seen[-1] == TIMEOUT or all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        wl.set_wait_limit(0)
    assert TIMEOUT in seen, seen
    got = call()
    done()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def case(M, K, N, r):
    g = torch.Generator(device="cuda").manual_seed(M)

    def normal(scale, *shape):
        return (scale * torch.randn(*shape, generator=g, device="cuda")).bfloat16()

    s = 0.9 + 0.2 * torch.rand(N, generator=g, device="cuda")
    U, V = (normal(0.02, N, r), normal(0.02, K, r)) if r else (None, None)
    return normal(1, M, K), (*wl.quantize_fp8(normal(0.02, N, K), 128), s, U, V), normal(1e-3, M, N)


@pytest.mark.parametrize("M,K,N,r", [
    (4, 21504, 20000, 0), (16, 21504, 5376, 0), (600, 21504, 2000, 0),  # stream: cut tiles, clusters; GEMM
    (16, 21504, 5376, 256), (4, 21504, 20000, 256), (600, 21504, 2000, 256)])
def test_forward_gives_up(M, K, N, r):
    x, p, _ = case(M, K, N, r)
    must_expire(lambda: wl.stacked_forward_fp8(x, [p]))


@pytest.mark.parametrize("M,N,K", [(16, 5376, 21504), (600, 2000, 21504)])
def test_product_gives_up(M, N, K):
    x, (codes, scales, *_), _ = case(M, K, N, 0)
    a = wl.quantize_fp8(x)
    must_expire(lambda: [wl.matmul_fp8(a, (codes, scales))])


@pytest.mark.parametrize("M,K,N", [(300, 1152, 20000), (8, 5376, 21504)])
def test_dx_gives_up(M, K, N):
    x, p, dy = case(M, K, N, 0)
    ckpt = wl.Fp8Checkpoint(*wl.quantize_fp8(x), [None])
    must_expire(lambda: [wl.stacked_backward_fp8(ckpt, [dy], [p], need_params=False)[0]])


@pytest.mark.parametrize("M,K,N", [(300, 21504, 2000), (8, 21504, 5376)])
def test_ds_gives_up(M, K, N):
    x, p, dy = case(M, K, N, 0)
    ckpt = wl.Fp8Checkpoint(*wl.quantize_fp8(x), [None])
    must_expire(lambda: [wl.stacked_backward_fp8(ckpt, [dy], [p], need_dx=False)[1][0][0]])


@pytest.mark.parametrize("what", ["dU", "dV"])
def test_rank_r_products_give_up(what):
    """dU alone (A by columns), and dV alone (E by rows, then A in 8 bits)."""
    M, K, N, r = 8192, 2048, 8192, 256
    x, (codes, scales, s, U, V), dy = case(M, K, N, r)
    xc, xs = wl.quantize_fp8(x)
    T = x @ V
    out = torch.empty(N if what == "dU" else K, r, dtype=torch.bfloat16, device="cuda")
    arr = (wl._GradFp8 * 1)(wl._GradFp8(*(t.data_ptr() for t in (codes, scales, s, U, V, T, dy)), None,
                                        *((out.data_ptr(), None) if what == "dU" else (None, out.data_ptr())), N, r))
    n = wl.lib().wl_stacked_backward_fp8_workspace(M, K, arr, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call():
        assert wl.lib().wl_stacked_backward_fp8(xc.data_ptr(), xs.data_ptr(), M, K, arr, 1, None, ws.data_ptr(), n, stream) == 0
        return [out]

    must_expire(call)
