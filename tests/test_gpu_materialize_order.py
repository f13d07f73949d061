"""GPU test of a rebuilt weight in use: the dense forward may directly follow
the kernel that rebuilds its weight."""
import pytest
import torch

import linear_wl_forward_b200 as wl
import wl_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,r", [(700, 520, 24), (4096, 1152, 64), (1152, 4096, 256)])
def test_forward_directly_behind_the_rebuild(N, K, r):
    call = wl_inputs.random_case(430 + N, 1, N, K, r)
    p = call.projs[0]
    bundle = [t.cuda() for t in (p.W0, p.s, p.U, p.V)]
    x, ones = call.x.cuda(), torch.ones(N, device="cuda")
    W = wl.materialize_weight(*bundle)
    torch.cuda.synchronize()
    want = wl.linear_forward(x, W, ones, None, None)
    y = torch.empty_like(want)
    for _ in range(10):
        W.zero_()
        y.zero_()
        torch.cuda.synchronize()
        wl.materialize_weight(*bundle, out=W)
        wl.linear_forward(x, W, ones, None, None, y=y)
        torch.cuda.synchronize()
        assert wl.last_device_status() == 0
        assert torch.equal(y, want)
