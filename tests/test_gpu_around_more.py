"""More of the operators around the block against the fp64 oracle (bounds as in
test_gpu_around.py)."""

import pytest

from tests.gpu_util import f64, have_gpu
from tests.test_gpu_around import Linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zb():
    if not have_gpu():
        pytest.skip("no CUDA device")
    from split_backward_gemms_gb300 import build as B
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


# the kernel for few rows or tiles, and the other one
@pytest.mark.parametrize("M,N,K", [(5, 64, 512), (60, 1032, 520), (300, 512, 4096), (300, 1032, 520), (2051, 2056, 264)])
@pytest.mark.parametrize("tanh", [False, True])
def test_gelu_keeps_h_in_the_residuals_place(zb, M, N, K, tanh):
    c = Linear(zb, M, N, K, "gelu", tanh=tanh)
    R = f64(c.R)
    c.kept = c.R
    c.run().check(R)
