"""CPU tests of the 8-bit operators' refusals: workspaces of refused sizes, and
arguments that are no tensors."""
import pytest
import torch

import linear_wl_forward_b200 as wl
from linear_wl_forward_b200 import build as wlbuild


@pytest.fixture(scope="module")
def L():
    wlbuild.build()
    return wl.lib()


def test_refused_products_need_no_workspace(L):
    top = (1 << 31) - 1
    for M, N, K in ((3, top, 4096), (3, 40000, top), (top, 40000, 4096), (3, 40000, top - 15), (3, 40000, 4104),
                    (-1, 40000, 4096), (3, -1, 4096), (3, 40000, -16), (3, (1 << 30) + 1, 4096)):
        assert L.wl_matmul_fp8_workspace(M, N, K) == 0, (M, N, K)
    assert L.wl_matmul_fp8_workspace(3, 40000, 4096) > 0


def test_none_where_a_tensor_is_needed():
    with pytest.raises(TypeError, match="T must be a CUDA tensor"):
        wl._ptr_on(torch.device("cuda", 0), None, torch.bfloat16, "T", (3, 8))
