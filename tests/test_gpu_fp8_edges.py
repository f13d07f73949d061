"""GPU tests of 8-bit calls at the edges of what their kernels' plans cover."""
import pytest

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
