"""CPU tests of the 8-bit operators: pins of their oracle, and what the C ABI
refuses on the host before it touches CUDA."""
import ctypes

import numpy as np
import pytest
import torch

import linear_wl_forward_b200 as wl
from linear_wl_forward_b200 import build as wlbuild
from oracle import fp8


@pytest.fixture(scope="module")
def L():
    wlbuild.build()
    return wl.lib()


# ------------------------------------------------------------------ oracle ----
def test_e4m3_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp8.e4m3_decode(codes), want)
    grid = fp8.e4m3_decode(np.arange(127))
    v = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, np.random.default_rng(0).uniform(0, 448, 4000),
                        np.exp2(np.random.default_rng(1).uniform(-14, 8, 4000))]).astype(np.float32)
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(fp8.e4m3_encode(v), want)
    assert fp8.e4m3_encode([np.nan, np.inf, -np.inf]).tolist() == [0x7F] * 3


def test_quantize_properties():
    rng = np.random.default_rng(2)
    a = rng.standard_normal((300, 272)) * np.exp2(rng.integers(-40, 40, (300, 1)))
    for rows in (1, 128):
        codes, scales = fp8.quantize(a, rows)
        assert scales.shape == (-(-300 // rows), 4) and (scales[:, 3:] == 127).all()
        back = fp8.dequantize(codes, scales, rows)
        S = np.exp2(scales.astype(np.float64) - 127)[np.arange(300) // rows][:, np.arange(272) // 128]
        # half a step: 2^-4 of a normal value, half of 2^-9 of the scale below
        assert (np.abs(back - a) <= np.maximum(np.abs(a) * 2.0 ** -4, S * 2.0 ** -10)).all()
        # the largest magnitude of each block lands above half of the range
        top = np.abs(fp8.e4m3_decode(codes[:128, :128])).max()
        assert 224 <= top <= 448
    codes, scales = fp8.quantize(np.zeros((2, 16)), 1)
    assert not codes.any() and (scales == 127).all()
    codes, scales = fp8.quantize(np.full((1, 16), 448.0), 1)
    assert scales[0, 0] == 127 and (codes == 126).all()
    codes, scales = fp8.quantize(np.full((1, 16), 449.0), 1)
    assert scales[0, 0] == 128


def test_oracle_forward_and_backward_by_hand():
    """Values that 8 bits hold exactly: the operators are those of exact
    arithmetic, and the gradients are checked against differences."""
    rng = np.random.default_rng(3)
    M, K, N, r = 5, 32, 7, 8
    x = rng.integers(-3, 4, (M, K)).astype(float)
    W = rng.integers(-2, 3, (N, K)).astype(float)
    s = np.exp2(rng.integers(-1, 2, N))
    U, V = rng.integers(-1, 2, (N, r)).astype(float), rng.integers(-1, 2, (K, r)).astype(float)
    dy = rng.integers(-2, 3, (M, N)).astype(float)

    def f(x, s, U, V):
        return sum(((s[n] * sum(W[n, k] * x[m, k] for k in range(K))
                     + sum(U[n, j] * sum(V[k, j] * x[m, k] for k in range(K)) for j in range(r))) * dy[m, n])
                   for m in range(M) for n in range(N))

    codes, scales = fp8.quantize(W, 128)
    (y, _), (T, _) = fp8.forward(x, codes, scales, s, U, V)
    np.testing.assert_array_equal(y, s * (x @ W.T) + (x @ V) @ U.T)
    np.testing.assert_array_equal(T, x @ V)
    xc, xs = fp8.quantize(x, 1)
    (dx, _), [((ds, _), (dU, _), (dV, _))] = fp8.backward(xc, xs, [dy], [T], [(codes, scales, s, U, V)])
    base = f(x, s, U, V)
    for name, arg, grad in (("x", x, dx), ("s", s, ds), ("U", U, dU), ("V", V, dV)):
        for _ in range(6):
            at = tuple(rng.integers(0, d) for d in arg.shape)
            moved = {"x": x, "s": s, "U": U, "V": V}
            moved[name] = arg.copy()
            moved[name][at] += 1  # f is linear in each argument
            assert f(**moved) - base == grad[at], (name, at)


# ---------------------------------------------------------------- refusals ----
A = 1 << 20  # 16-byte aligned stand-in address; never dereferenced
INVALID, ALIGN, UNSUPPORTED = 1, 2, 3


def test_quantize_refusals(L):
    def q(a=A, type=0, rows=4, cols=32, block=1, codes=A, scales=A):
        return L.wl_quantize_fp8(a, type, rows, cols, block, codes, scales, None)

    assert q(a=None) == q(codes=None) == q(scales=None) == INVALID
    assert q(type=2) == q(block=64) == q(rows=-1) == q(cols=-16) == INVALID
    assert q(cols=24) == q(a=A + 8) == q(codes=A + 8) == q(scales=A + 2) == ALIGN
    assert q(rows=0, a=None, codes=None, scales=None) == 0 and q(cols=0) == 0
    assert q(cols=(1 << 30) + 16) == UNSUPPORTED


def test_matmul_refusals(L):
    def m(ac=A, asc=A, bc=A, bsc=A, y=A, M=200, N=40, K=64, ws=A, n=1 << 30):
        return L.wl_matmul_fp8(ac, asc, bc, bsc, y, M, N, K, ws, n, None)

    assert m(ac=None) == m(asc=None) == m(bc=None) == m(bsc=None) == m(y=None) == INVALID
    assert m(M=-1) == m(N=-1) == m(K=-16) == INVALID
    assert m(K=40) == m(ac=A + 8) == m(bc=A + 4) == m(asc=A + 2) == m(bsc=A + 1) == m(y=A + 1) == ALIGN
    assert m(M=0) == m(N=0) == 0
    need = L.wl_matmul_fp8_workspace(3, 40000, 4096)
    assert need > 0
    assert m(M=3, N=40000, K=4096, n=need - 1) == m(M=3, N=40000, K=4096, ws=None) == INVALID
    assert m(M=3, N=40000, K=4096, ws=A + 8, n=need) == ALIGN


def proj(**kw):
    v = dict(codes=A, scales=A, s=A, U=A, V=A, y=A, T=None, N=40, r=8)
    v.update(kw)
    return wl._ProjFp8(*v.values())


def grad(**kw):
    v = dict(codes=A, scales=A, s=A, U=A, V=A, T=A, dy=A, ds=A, dU=A, dV=A, N=40, r=8)
    v.update(kw)
    return wl._GradFp8(*v.values())


def test_forward_refusals(L):
    def f(*ps, x=A, M=3, K=64, xc=None, xs=None, ws=A, n=1 << 30, P=None):
        ps = ps or (proj(),)
        arr = (wl._ProjFp8 * max(len(ps), 1))(*ps)
        args = (x, M, K, arr, len(ps) if P is None else P, xc, xs, ws, n)
        code = L.wl_stacked_forward_fp8(*args, None)
        plan = ctypes.c_void_p()
        assert L.wl_plan_stacked_forward_fp8(*args, ctypes.byref(plan)) == code and (code == 0) == bool(plan.value)
        return code

    assert f(x=None) == f(proj(codes=None)) == f(proj(scales=None)) == f(proj(s=None)) == f(proj(y=None)) == INVALID
    assert f(proj(U=None)) == f(proj(V=None)) == f(M=-1) == f(K=-16) == f(proj(N=-1)) == f(proj(r=-8)) == INVALID
    assert f(xc=A) == f(xs=A) == f(P=0) == f(n=64) == f(ws=None) == INVALID
    assert L.wl_stacked_forward_fp8(A, 3, 64, None, 1, None, None, A, 1 << 30, None) == INVALID
    assert f(P=9) == f(proj(r=1032)) == f(proj(N=(1 << 30) + 1)) == f(K=(1 << 30) + 16) == UNSUPPORTED
    assert f(K=72) == f(proj(r=12)) == f(x=A + 8) == f(proj(codes=A + 8)) == f(proj(scales=A + 2)) == ALIGN
    assert f(proj(U=A + 8)) == f(proj(V=A + 2)) == f(proj(T=A + 4)) == f(proj(y=A + 1)) == f(proj(s=A + 2)) == ALIGN
    assert f(xc=A + 8, xs=A) == f(xc=A, xs=A + 1) == f(ws=A + 8) == ALIGN
    assert L.wl_plan_stacked_forward_fp8(A, 3, 64, (wl._ProjFp8 * 1)(proj()), 1, None, None, A, 1 << 30, None) == INVALID
    assert L.wl_run_fp8_plan(None, None) == INVALID
    L.wl_free_fp8_plan(None)


def test_backward_refusals(L):
    def b(*ps, xc=A, xs=A, M=3, K=64, dx=A, ws=A, n=1 << 30, P=None):
        ps = ps or (grad(),)
        return L.wl_stacked_backward_fp8(xc, xs, M, K, (wl._GradFp8 * len(ps))(*ps), len(ps) if P is None else P, dx, ws, n, None)

    assert b(xc=None) == b(xs=None) == b(grad(dy=None)) == b(grad(s=None)) == b(grad(codes=None)) == INVALID
    assert b(grad(U=None)) == b(grad(V=None)) == b(grad(T=None)) == b(M=-1) == b(K=-16) == b(P=0) == b(n=8) == INVALID
    assert b(P=9) == b(grad(r=1032)) == UNSUPPORTED
    assert b(K=8) == b(grad(r=4)) == b(xc=A + 8) == b(dx=A + 8) == b(grad(dU=A + 8)) == b(grad(dV=A + 2)) == ALIGN
    assert b(grad(dy=A + 1)) == b(grad(ds=A + 2)) == b(grad(T=A + 8)) == b(ws=A + 4) == ALIGN


def test_workspace_sizes(L):
    arr = (wl._ProjFp8 * 2)(proj(N=300, r=16), proj(N=40, r=0))
    sizes = [L.wl_stacked_forward_fp8_workspace(M, 528, arr, 2) for M in (0, 1, 64, 200, 1000)]
    assert sizes[0] == 0 and all(s > 0 for s in sizes[1:])
    assert sizes[4] >= 1000 * 528
    assert L.wl_stacked_forward_fp8_workspace(8, 520, arr, 2) == 0  # refused sizes
    arr = (wl._GradFp8 * 1)(grad(N=300, r=16))
    assert L.wl_stacked_backward_fp8_workspace(64, 528, arr, 1) >= 64 * 304


def test_python_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    for call in (lambda: wl.quantize_fp8(x), lambda: wl.stacked_forward_fp8(x, []), lambda: wl.prepare_stacked_fp8(x, []),
                 lambda: wl.matmul_fp8((x, x), (x, x)),
                 lambda: wl.stacked_backward_fp8(wl.Fp8Checkpoint(x, x, []), [], [])):
        with pytest.raises(TypeError):
            call()
    assert [wl.fp8_scale_pitch(c) for c in (0, 16, 512, 528)] == [0, 4, 4, 8]
