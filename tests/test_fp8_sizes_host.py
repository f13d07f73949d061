"""CPU tests of the 8-bit operators' sizes: workspaces of calls that are refused."""
import pytest

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
