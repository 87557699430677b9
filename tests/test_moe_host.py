"""Refusals of the mixture-of-experts and 8-bit entry points (no GPU: every
error is returned before any device work), and the oracle's own checks."""

import ctypes as C

import numpy as np
import pytest

from oracle import moe as om
from split_backward_gemms_gb300 import build as B

P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def zb():
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


def refused(zb, status, call, *args, **kw):
    with pytest.raises(zb.ZBError) as e:
        call(*args, **kw)
    assert e.value.status == status, str(e.value)
    assert zb.zb_last_error()


@pytest.mark.parametrize("field,value,status", [
    ("experts", 0, "SHAPE"), ("experts", 257, "SHAPE"), ("topk", 0, "SHAPE"), ("topk", 9, "SHAPE"),
    ("topk", 33, "SHAPE"), ("tokens", -1, "SHAPE"), ("tokens", 1 << 30, "SHAPE"), ("dtype", 5, "DTYPE"),
    ("renorm", 2, "INVALID_ARG")])
def test_router_refuses(zb, field, value, status):
    r = zb.make_router(4, 8, 2)
    setattr(r, field, value)
    code = getattr(zb, "ZB_ERR_" + status)
    refused(zb, code, zb.zb_moe_route, r, P, P, P, P, P, P, P, 1 << 20, stream=0)
    if field != "tokens" or value:
        refused(zb, code, zb.zb_moe_route_backward, r, P, P, P, P, P, stream=0)
    assert zb.zb_moe_route_workspace_bytes(r) == 0


def test_route_refuses_pointers(zb):
    r = zb.make_router(4, 8, 2)
    n = zb.zb_moe_route_workspace_bytes(r)
    good = [P] * 7
    for i in range(6):
        refused(zb, zb.ZB_ERR_INVALID_ARG, zb.zb_moe_route, r, *[None if j == i else p for j, p in enumerate(good)], n,
                stream=0)
    for i in range(7):
        refused(zb, zb.ZB_ERR_ALIGN, zb.zb_moe_route, r, *[p + 4 if j == i else p for j, p in enumerate(good)], n,
                stream=0)
    refused(zb, zb.ZB_ERR_WORKSPACE, zb.zb_moe_route, r, *good, n - 1, stream=0)
    refused(zb, zb.ZB_ERR_WORKSPACE, zb.zb_moe_route, r, *good[:6], None, n, stream=0)
    for renorm in (0, 1):
        r.renorm = renorm
        for i in range(0 if not renorm else 1, 5):
            refused(zb, zb.ZB_ERR_INVALID_ARG, zb.zb_moe_route_backward, r,
                    *[None if j == i else P for j in range(5)], stream=0)


def test_rows_refuse(zb):
    calls = [(zb.zb_moe_dispatch, 3), (zb.zb_moe_combine, 4), (zb.zb_moe_combine_backward, 6)]
    for call, n in calls:
        refused(zb, zb.ZB_ERR_SHAPE, call, 4, 0, 64, *[P] * n, stream=0)
        refused(zb, zb.ZB_ERR_SHAPE, call, 4, 33, 64, *[P] * n, stream=0)
        refused(zb, zb.ZB_ERR_SHAPE, call, -1, 2, 64, *[P] * n, stream=0)
        refused(zb, zb.ZB_ERR_SHAPE, call, 1 << 30, 2, 64, *[P] * n, stream=0)
        refused(zb, zb.ZB_ERR_SHAPE, call, 4, 2, 0, *[P] * n, stream=0)
        refused(zb, zb.ZB_ERR_ALIGN, call, 4, 2, 60, *[P] * n, stream=0)
        for i in range(n):
            if call is zb.zb_moe_combine and i == 2:
                continue  # gates may be NULL
            refused(zb, zb.ZB_ERR_INVALID_ARG, call, 4, 2, 64, *[None if j == i else P for j in range(n)], stream=0)
        refused(zb, zb.ZB_ERR_ALIGN, call, 4, 2, 64, P + 8, *[P] * (n - 1), stream=0)


@pytest.mark.parametrize("field,value,status", [
    ("experts", 0, "SHAPE"), ("experts", 257, "SHAPE"), ("rows", -1, "SHAPE"), ("rows", (1 << 30) + 1, "SHAPE"),
    ("h", 0, "SHAPE"), ("f", 0, "SHAPE"), ("h", 12, "ALIGN"), ("f", 20, "ALIGN"), ("act", 3, "INVALID_ARG"),
    ("flags", 1, "INVALID_ARG"), ("has_bias", 2, "INVALID_ARG")])
def test_experts_refuse(zb, field, value, status):
    m = zb.make_moe(16, 64, 128, 4)
    setattr(m, field, value)
    code = getattr(zb, "ZB_ERR_" + status)
    refused(zb, code, zb.zb_moe_forward, m, *[P] * 9, stream=0)
    refused(zb, code, zb.zb_moe_backward_input, m, *[P] * 7, stream=0)
    refused(zb, code, zb.zb_moe_backward_weight, m, *[P] * 9, 0, P, 1 << 20, stream=0)
    assert zb.zb_moe_workspace_bytes(m) == 0


def test_experts_refuse_pointers(zb):
    m = zb.make_moe(16, 64, 128, 4, has_bias=True)
    n = zb.zb_moe_workspace_bytes(m)
    for call, k in ((zb.zb_moe_forward, 9), (zb.zb_moe_backward_input, 7)):
        for i in range(k):
            refused(zb, zb.ZB_ERR_INVALID_ARG, call, m, *[None if j == i else P for j in range(k)], stream=0)
            refused(zb, zb.ZB_ERR_ALIGN, call, m, *[P + 2 if j == i else P for j in range(k)], stream=0)
    for i in range(9):
        refused(zb, zb.ZB_ERR_INVALID_ARG, zb.zb_moe_backward_weight, m, *[None if j == i else P for j in range(9)], 0,
                P, n, stream=0)
        refused(zb, zb.ZB_ERR_ALIGN, zb.zb_moe_backward_weight, m, *[P + 2 if j == i else P for j in range(9)], 0, P, n,
                stream=0)
    refused(zb, zb.ZB_ERR_WORKSPACE, zb.zb_moe_backward_weight, m, *[P] * 9, 0, P, n - 1, stream=0)
    refused(zb, zb.ZB_ERR_WORKSPACE, zb.zb_moe_backward_weight, m, *[P] * 9, 0, None, n, stream=0)
    refused(zb, zb.ZB_ERR_ALIGN, zb.zb_moe_backward_weight, m, *[P] * 9, 0, P + 128, n, stream=0)


def test_fp8_refuses(zb):
    q, w = zb.zb_fp8_quantize_rows, zb.zb_fp8_quantize_weight
    refused(zb, zb.ZB_ERR_SHAPE, q, -1, 16, P, P, P, stream=0)
    refused(zb, zb.ZB_ERR_SHAPE, q, 4, 0, P, P, P, stream=0)
    refused(zb, zb.ZB_ERR_ALIGN, q, 4, 24, P, P, P, stream=0)
    refused(zb, zb.ZB_ERR_ALIGN, q, 4, 16, P + 8, P, P, stream=0)
    refused(zb, zb.ZB_ERR_INVALID_ARG, q, 4, 16, P, None, P, stream=0)
    refused(zb, zb.ZB_ERR_SHAPE, w, 0, 16, 16, P, P, P, P, P, stream=0)
    refused(zb, zb.ZB_ERR_SHAPE, w, 257, 16, 16, P, P, P, P, P, stream=0)
    refused(zb, zb.ZB_ERR_ALIGN, w, 1, 24, 16, P, P, P, P, P, stream=0)
    refused(zb, zb.ZB_ERR_INVALID_ARG, w, 1, 16, 16, P, P, None, P, P, stream=0)
    refused(zb, zb.ZB_ERR_INVALID_ARG, w, 1, 16, 16, P, None, None, None, None, stream=0)
    g = zb.make_fp8_matmul(4, 64, 32, experts=2)
    good = [P] * 8  # offsets, Xq, xs, Wq, ws, H, out0, out1
    for i in (0, 1, 2, 3, 4, 6):
        refused(zb, zb.ZB_ERR_INVALID_ARG, zb.zb_fp8_matmul, g, *[None if j == i else p for j, p in enumerate(good)],
                stream=0)
    refused(zb, zb.ZB_ERR_ALIGN, zb.zb_fp8_matmul, g, P, P + 8, *good[2:], stream=0)
    for epi, missing in ((zb.ZB_FP8_GELU, 7), (zb.ZB_FP8_GELU_GRAD, 5)):
        g.epilogue = epi
        refused(zb, zb.ZB_ERR_INVALID_ARG, zb.zb_fp8_matmul, g,
                *[None if j == missing else p for j, p in enumerate(good)], stream=0)
    refused(zb, zb.ZB_ERR_INVALID_ARG, zb.zb_fp8_matmul, g, *good, bias=P, stream=0)
    for field, value, status in (("K", 24, "ALIGN"), ("N", 12, "ALIGN"), ("M", -1, "SHAPE"), ("K", 0, "SHAPE"),
                                 ("N", 0, "SHAPE"), ("experts", 0, "SHAPE"), ("experts", 300, "SHAPE"),
                                 ("epilogue", 3, "INVALID_ARG"), ("act", 0, "INVALID_ARG"),
                                 ("scales", 2, "INVALID_ARG")):
        g = zb.make_fp8_matmul(4, 64, 32, experts=2, epilogue=zb.ZB_FP8_GELU)
        setattr(g, field, value)
        refused(zb, getattr(zb, "ZB_ERR_" + status), zb.zb_fp8_matmul, g, *good, stream=0)


def test_descriptor_sizes(zb):
    assert C.sizeof(zb.zb_router) == 24 and C.sizeof(zb.zb_moe) == 40 and C.sizeof(zb.zb_fp8_gemm) == 40


def test_oracle_e4m3_is_the_nearest_value():
    """Against the list of every e4m3 value, ties to the even mantissa."""
    grid = [m * 2.0 ** -9 for m in range(8)]
    grid += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if not (e == 8 and m == 7)]
    grid = np.array(sorted(set(grid)))
    assert grid.max() == 448.0 and len(grid) == 127
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(0, 448, 500), np.exp2(rng.uniform(-12, 8.8, 500)), (grid[1:] + grid[:-1]) / 2])
    for v in x:
        d = np.abs(grid - v)
        best = np.flatnonzero(d == d.min())
        want = grid[[b for b in best if b % 2 == 0][0]] if len(best) == 2 else grid[best[0]]
        assert om.e4m3(v) == want and om.e4m3(-v) == -want


def test_oracle_scale():
    for amax in (448.0, 448.0001, 1.0, 1.75, 1.7500001, 3e38, 1e-45, 2.0 ** -120):
        s = om.block_scale(amax)
        assert amax / s <= 448.0 and (amax / (s / 2) > 448.0 or s == 2.0 ** -126)
    assert om.block_scale(0.0) == 1.0 and np.isnan(om.block_scale(np.inf)) and np.isnan(om.block_scale(np.nan))


def test_route_backward_by_differences():
    """The oracle's gradient formula against central differences of its gates."""
    rng = np.random.default_rng(2)
    for renorm in (False, True):
        z = rng.normal(size=(3, 6))
        dg = rng.normal(size=(3, 2))
        _, expert, *_ = om.route(z, 2, renorm)
        grad = om.route_backward(z, expert, dg, renorm)
        for t in range(3):
            for i in range(6):
                d = np.zeros_like(z)
                d[t, i] = 1e-6
                up, down = om.route(z + d, 2, renorm)[0], om.route(z - d, 2, renorm)[0]
                assert abs(((up - down) * dg).sum() / 2e-6 - grad[t, i]) < 1e-8


@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_layer_gradients_by_differences(renorm):
    """Router, dispatch, experts, combine: every gradient against central
    differences of the layer's output (choices do not change at these steps)."""
    rng = np.random.default_rng(3)
    T, E, k, h, f = 5, 4, 2, 3, 4
    X, z = rng.normal(size=(T, h)), rng.normal(size=(T, E))
    W1, W2, dout = rng.normal(size=(E, h, f)), rng.normal(size=(E, f, h)), rng.normal(size=(T, h))
    _, s = om.layer_forward(X, z, k, renorm, W1, W2)
    grads = om.layer_backward(dout, z, renorm, W1, W2, s)
    args = [X, z, W1, W2]

    def value():
        return (om.layer_forward(args[0], args[1], k, renorm, args[2], args[3])[0] * dout).sum()

    for a, g in zip(args, grads):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 1e-6
            up = value()
            a[i] = old - 1e-6
            down = value()
            a[i] = old
            # central differences: O(step^2) plus rounding of the values over the step
            assert abs((up - down) / 2e-6 - g[i]) < 1e-7 * max(1.0, abs(g[i]))
