"""The example's mixture-of-experts stage against the oracle's layer.

The stage rounds to bf16 at its storage points (rows, H, A, Y, dY, dH, dX);
the oracle does not, so gradients are compared in relative Frobenius norm at
2e-2, the figure of the other unrounded chains; with 8-bit products each
operand's rounding is up to 2^-4 relative (3 mantissa bits), about 2.6 % in the
norm for each of the two to four products of a chain: 1.5e-1.
"""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import moe as om
from tests.gpu_util import f64, have_gpu, sync

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not have_gpu():
        pytest.skip("no CUDA device")
    from split_backward_gemms_gb300 import build as B
    B.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_stage
    return moe_stage


def rel(a, b):
    return np.linalg.norm(f64(a) - b) / np.linalg.norm(b)


@pytest.mark.parametrize("fp8,tol", [(False, 2e-2), (True, 1.5e-1)])
@pytest.mark.parametrize("T,E,k,h,f", [(70, 4, 2, 128, 256), (333, 16, 4, 144, 272)])
def test_stage_against_oracle(ex, fp8, tol, T, E, k, h, f):
    rng = np.random.default_rng(T)

    def dev(a, dtype=torch.bfloat16):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype).cuda()

    m = 2
    st = ex.Stage(T, h, f, E, k, m, fp8=fp8)
    W1, W2 = dev(rng.normal(size=(E, h, f)) / np.sqrt(h)), dev(rng.normal(size=(E, f, h)) / np.sqrt(f))
    st.set_weights(W1, W2)
    sums = [np.zeros(W1.shape), np.zeros(W2.shape)]
    for j in range(m):
        X, z, dout = dev(rng.normal(size=(T, h))), dev(rng.normal(size=(T, E)), torch.float32), dev(rng.normal(size=(T, h)))
        z[:3] = -float("inf")  # padding tokens
        out = st.forward(j, X, z)
        din = st.backward_input(j, dout)
        sync(ex.zb)
        ref, s = om.layer_forward(f64(X), f64(z), k, True, f64(W1), f64(W2))
        dX, dz, dW1, dW2 = om.layer_backward(f64(dout), f64(z), True, f64(W1), f64(W2), s)
        assert rel(out, ref) < tol and rel(din, dX) < tol and rel(st.micro[j]["dlogits"], dz) < tol
        assert (out[:3] == 0).all() and (din[:3] == 0).all()
        sums[0] += dW1
        sums[1] += dW2
    for j in range(m):
        st.backward_weight(j)
    sync(ex.zb)
    assert rel(st.dW1, sums[0]) < tol and rel(st.dW2, sums[1]) < tol


@pytest.mark.parametrize("fp8", [False, True])
def test_example_learns(ex, fp8, monkeypatch, capsys):
    argv = ["moe_stage.py", "--steps", "10", "--tokens", "256", "--h", "128", "--f", "256", "--micro", "2"]
    monkeypatch.setattr(sys, "argv", argv + (["--fp8"] if fp8 else []))
    losses = ex.main()
    assert losses[-1] < 0.8 * losses[0]
