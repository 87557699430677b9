"""Refusals of the linear, layer-norm and embedding entry points (no GPU: every
error is returned before any device work), and the oracle's own checks."""

import ctypes as C

import numpy as np
import pytest

from oracle import around as oa
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
    assert e.value.status == getattr(zb, "ZB_ERR_" + status), str(e.value)
    assert zb.zb_last_error()


def without(args, i, by=None):
    return [by if j == i else a for j, a in enumerate(args)]


# ------------------------------------------------------------------- linear
@pytest.mark.parametrize("field,value,status", [
    ("M", -1, "SHAPE"), ("M", (1 << 30) + 1, "SHAPE"), ("N", 0, "SHAPE"), ("N", -8, "SHAPE"), ("N", 1 << 31, "SHAPE"),
    ("K", 0, "SHAPE"), ("K", 1 << 31, "SHAPE"), ("N", 60, "ALIGN"), ("K", 36, "ALIGN"), ("transposed", 2, "INVALID_ARG"),
    ("transposed", -1, "INVALID_ARG"), ("epilogue", 3, "INVALID_ARG"), ("epilogue", -1, "INVALID_ARG"),
    ("dtype", 2, "DTYPE"), ("ldx", 24, "SHAPE"), ("ldw", 56, "SHAPE"), ("ldr", 56, "SHAPE"), ("ldh", -64, "SHAPE"),
    ("ldo", 8, "SHAPE"), ("ldo", 1 << 31, "SHAPE"), ("ldx", 36, "ALIGN"), ("ldw", 68, "ALIGN"), ("ldr", 65, "ALIGN"),
    ("ldh", 66, "ALIGN"), ("ldo", 68, "ALIGN")])
def test_linear_refuses(zb, field, value, status):
    g = zb.make_linear(16, 64, 32)
    setattr(g, field, value)
    refused(zb, status, zb.zb_linear_product, g, P, P, P, P, None, P, None, stream=0)


def test_linear_refuses_forms(zb):
    for form in (zb.ZB_LINEAR_GELU, zb.ZB_LINEAR_GELU_GRAD):
        bias = P if form == zb.ZB_LINEAR_GELU else None
        for act in (zb.ZB_ACT_NONE, 3, -1):
            g = zb.make_linear(16, 64, 32, epilogue=form, act=act)
            refused(zb, "INVALID_ARG", zb.zb_linear_product, g, P, P, bias, P, P, P, P, stream=0)
        g = zb.make_linear(16, 64, 32, epilogue=form, dtype=zb.ZB_DT_F32)
        refused(zb, "DTYPE", zb.zb_linear_product, g, P, P, bias, P, P, P, P, stream=0)
    g = zb.make_linear(16, 64, 32, epilogue=zb.ZB_LINEAR_GELU_GRAD)
    refused(zb, "INVALID_ARG", zb.zb_linear_product, g, P, P, P, P, P, P, None, stream=0)  # bias
    # a transposed weight's rows have K values
    g = zb.make_linear(16, 64, 128, transposed=True, ldw=64)
    refused(zb, "SHAPE", zb.zb_linear_product, g, P, P, None, None, None, P, None, stream=0)


def test_linear_refuses_pointers(zb):
    good = [P] * 7  # X, W, bias, R, H, out0, out1
    for form, needs in ((zb.ZB_LINEAR_STORE, (0, 1, 5)), (zb.ZB_LINEAR_GELU, (0, 1, 6)),
                        (zb.ZB_LINEAR_GELU_GRAD, (0, 1, 4, 5))):
        g = zb.make_linear(16, 64, 32, epilogue=form)
        args = without(good, 2) if form == zb.ZB_LINEAR_GELU_GRAD else good
        for i in needs:
            refused(zb, "INVALID_ARG", zb.zb_linear_product, g, *without(args, i), stream=0)
        for i in range(7):
            if args[i] is not None:
                refused(zb, "ALIGN", zb.zb_linear_product, g, *without(args, i, P + 8), stream=0)


# --------------------------------------------------------------------- norm
@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, "SHAPE"), ("rows", (1 << 30) + 1, "SHAPE"), ("width", 0, "SHAPE"), ("width", 32776, "SHAPE"),
    ("width", 12, "ALIGN"), ("dtype", 2, "DTYPE"), ("dtype", -1, "DTYPE"), ("eps", 0.0, "INVALID_ARG"),
    ("eps", -1e-5, "INVALID_ARG"), ("eps", float("nan"), "INVALID_ARG"), ("eps", float("inf"), "INVALID_ARG")])
def test_norm_refuses(zb, field, value, status):
    n = zb.make_layernorm(4, 64)
    setattr(n, field, value)
    refused(zb, status, zb.zb_layernorm_forward, n, *[P] * 6, stream=0)
    refused(zb, status, zb.zb_layernorm_backward_input, n, *[P] * 8, stream=0)
    refused(zb, status, zb.zb_layernorm_backward_weight, n, *[P] * 6, 0, stream=0)


def test_norm_refuses_pointers(zb):
    n = zb.make_layernorm(4, 64)
    calls = [(zb.zb_layernorm_forward, 6, (0, 1, 3, 4, 5), (0, 1, 2, 3), ()),
             (zb.zb_layernorm_backward_input, 8, (0, 1, 2, 3, 4, 6), (0, 1, 2, 5, 6, 7), ()),
             (zb.zb_layernorm_backward_weight, 6, (0, 1, 2, 3, 4), (0, 1), (0,))]
    for call, k, needs, wide, more in calls:
        for i in range(k):
            if i in needs:  # mean without rstd, or the other way round, too
                refused(zb, "INVALID_ARG", call, n, *without([P] * k, i), *more, stream=0)
            refused(zb, "ALIGN", call, n, *without([P] * k, i, P + (8 if i in wide else 2)), *more, stream=0)


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("field,value,status", [
    ("tokens", -1, "SHAPE"), ("tokens", (1 << 30) + 1, "SHAPE"), ("vocab", 0, "SHAPE"), ("vocab", 1 << 31, "SHAPE"),
    ("width", 0, "SHAPE"), ("width", (1 << 20) + 8, "SHAPE"), ("width", 20, "ALIGN"), ("dtype", 2, "DTYPE")])
def test_embedding_refuses(zb, field, value, status):
    e = zb.make_embedding(40, 100, 64)
    setattr(e, field, value)
    assert zb.zb_embedding_workspace_bytes(e) == 0
    refused(zb, status, zb.zb_embedding_forward, e, P, P, P, stream=0)
    refused(zb, status, zb.zb_embedding_sort, e, P, P, P, P, 1 << 20, stream=0)
    refused(zb, status, zb.zb_embedding_backward, e, P, P, P, P, 0, P, 1 << 20, stream=0)


@pytest.mark.parametrize("tokens", [40, 5000])
def test_embedding_refuses_pointers(zb, tokens):
    e = zb.make_embedding(tokens, 100, 64)
    n = zb.zb_embedding_workspace_bytes(e)
    assert n > 0 and n % 256 == 0
    for i in range(3):
        refused(zb, "INVALID_ARG", zb.zb_embedding_forward, e, *without([P] * 3, i), stream=0)
        refused(zb, "ALIGN", zb.zb_embedding_forward, e, *without([P] * 3, i, P + (8 if i else 2)), stream=0)
        refused(zb, "INVALID_ARG", zb.zb_embedding_sort, e, *without([P] * 3, i), P, n, stream=0)
        refused(zb, "ALIGN", zb.zb_embedding_sort, e, *without([P] * 3, i, P + 2), P, n, stream=0)
    for i in range(4):
        refused(zb, "INVALID_ARG", zb.zb_embedding_backward, e, *without([P] * 4, i), 0, P, n, stream=0)
        refused(zb, "ALIGN", zb.zb_embedding_backward, e, *without([P] * 4, i, P + (8 if i > 1 else 2)), 0, P, n,
                stream=0)
    for call, args in ((zb.zb_embedding_sort, [P] * 3), (zb.zb_embedding_backward, [P] * 4 + [0])):
        refused(zb, "WORKSPACE", call, e, *args, P, n - 1, stream=0)
        refused(zb, "WORKSPACE", call, e, *args, None, n, stream=0)
        refused(zb, "ALIGN", call, e, *args, P + 128, n, stream=0)


def test_nothing_to_do_needs_no_buffers(zb):
    """Empty calls return before any device work (here there is no device)."""
    zb.zb_linear_product(zb.make_linear(0, 64, 32), None, None, None, None, None, None, None, stream=0)
    n = zb.make_layernorm(0, 64)
    zb.zb_layernorm_forward(n, None, None, None, None, None, None, stream=0)
    zb.zb_layernorm_backward_input(n, None, None, None, None, None, None, None, None, stream=0)
    e = zb.make_embedding(0, 100, 64)
    assert zb.zb_embedding_workspace_bytes(e) == 0
    zb.zb_embedding_forward(e, None, None, None, stream=0)
    zb.zb_embedding_sort(e, None, None, None, None, 0, stream=0)
    zb.zb_embedding_backward(e, None, None, None, P, 1, None, 0, stream=0)


def test_descriptor_sizes(zb):
    assert C.sizeof(zb.zb_linear) == 80 and C.sizeof(zb.zb_layernorm) == 24 and C.sizeof(zb.zb_embedding) == 32


# ------------------------------------------------------------- the oracle's
def _difference(f, a, g, step=1e-6):
    """The gradient g of the scalar f() to the array a, against central differences."""
    for i in np.ndindex(a.shape):
        old = a[i]
        a[i] = old + step
        up = f()
        a[i] = old - step
        down = f()
        a[i] = old
        assert abs((up - down) / (2 * step) - g[i]) < 1e-7 * max(1.0, abs(g[i]))


def test_oracle_norm_gradients_by_differences():
    rng = np.random.default_rng(0)
    X, gamma, beta, dY = (rng.normal(size=s) for s in ((3, 5), 5, 5, (3, 5)))
    eps = 0.1

    def value():
        return (oa.norm_forward(X, gamma, beta, eps)[0] * dY).sum()

    _, mean, rstd = oa.norm_forward(X, gamma, beta, eps)
    dg, db = oa.norm_backward_weight(dY, X, mean, rstd)
    _difference(value, X, oa.norm_backward_input(dY, X, gamma, mean, rstd))
    _difference(value, gamma, dg)
    _difference(value, beta, db)


def test_oracle_embedding_gradient_by_differences():
    rng = np.random.default_rng(1)
    ids = [2, -1, 0, 2, 9, 4, 2]
    E, dY = rng.normal(size=(5, 3)), rng.normal(size=(7, 3))
    _difference(lambda: (oa.embedding(ids, E, 1.5) * dY).sum(), E, oa.embedding_backward(ids, 5, dY, 1.5))
    order, sid = oa.embedding_order(ids, 5)
    assert order.tolist() == [2, 0, 3, 6, 5, 1, 4] and sid.tolist() == [0, 2, 2, 2, 4, -1, -1]


@pytest.mark.parametrize("tanh", [False, True])
def test_oracle_block_gradients_by_differences(tanh):
    """R + GeLU(LN(R) W1 + b1) W2 + b2: the gradient of R through the norm and
    along the residual, put together from the operators' oracles."""
    rng = np.random.default_rng(2)
    T, h, f, eps = 3, 4, 5, 0.1
    R, W1, b1, W2, b2 = (rng.normal(size=s) for s in ((T, h), (h, f), f, (f, h), h))
    gamma, beta, dY = (rng.normal(size=s) for s in (h, h, (T, h)))

    def forward():
        N, mean, rstd = oa.norm_forward(R, gamma, beta, eps)
        A, H = oa.linear(N, W1, form="gelu", bias=b1, tanh=tanh)
        return oa.linear(A, W2, bias=b2, R=R)[0], (N, mean, rstd, A, H)

    _, (N, mean, rstd, A, H) = forward()
    dH, _ = oa.linear(dY, W2, transposed=True, form="grad", H=H, tanh=tanh)
    dN, _ = oa.linear(dH, W1, transposed=True)
    dR = oa.norm_backward_input(dN, R, gamma, mean, rstd, dR=dY)
    dg, db = oa.norm_backward_weight(dN, R, mean, rstd)
    f = lambda: (forward()[0] * dY).sum()  # noqa: E731
    _difference(f, R, dR)
    _difference(f, gamma, dg)
    _difference(f, beta, db)
    _difference(f, W1, N.T @ dH)
