"""GPU parity of the 8-bit products and their quantisers against the oracle.

The quantisers are exact but for e4m3's rounding, so their values and scales
equal the oracle's.  The products' bounds: as for the bf16 products (an e4m3
product is exact in fp32; a scaled partial sum adds one rounding for each block
of 128, inside the n 2^-23 bound).
"""

import numpy as np
import pytest
import torch

from oracle import moe as om
from tests.gpu_util import empty_bf16, empty_f32, f64, have_gpu, sync
from tests.test_gpu_moe import dev, i32, near

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn
NAN = float("nan")


@pytest.fixture(scope="module")
def zb():
    if not have_gpu():
        pytest.skip("no CUDA device")
    from split_backward_gemms_gb300 import build as B
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


def e4(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda").view(E4)


def values(q):
    return q.float().cpu().double().numpy()


def _rows(rng, R, K):
    """Values over many binades, with the edges of the scale's rule in some blocks."""
    X = rng.normal(size=(R, K)) * np.exp2(rng.integers(-30, 30, size=(R, 1)))
    flat = X.reshape(-1)
    for i, v in enumerate((448.0, 449.0, 450.0, 1.75, 1.7578125, 2.0 ** -9, 3e38, 1e-40, 2.0 ** -133)):
        if i < R:
            X[i, :] = 0.0
            X[i, i % K] = v
            X[i, (i + 3) % K] = -v / 2
    if R > 12:
        X[10] = 0.0  # a block of zeros
    del flat
    return X


@pytest.mark.parametrize("R,K", [(1, 16), (3, 128), (13, 144), (70, 1040), (257, 512)])
def test_quantize_rows(zb, R, K):
    X = dev(_rows(np.random.default_rng(R), R, K))
    Q, S = e4(R, K), empty_f32(R, -(-K // 128))
    zb.zb_fp8_quantize_rows(R, K, X, Q, S)
    sync(zb)
    q, s = om.quantize_rows(f64(X))
    assert np.array_equal(f64(S), s)
    assert np.array_equal(values(Q), q)


def test_quantize_marks_what_is_not_finite(zb):
    X = np.ones((3, 256))
    X[0, 5] = np.inf
    X[1, 200] = np.nan
    Q, S = e4(3, 256), empty_f32(3, 2)
    zb.zb_fp8_quantize_rows(3, 256, dev(X), Q, S)
    sync(zb)
    assert np.array_equal(np.isnan(f64(S)), [[True, False], [False, True], [False, False]])
    assert not np.isnan(values(Q)[2]).any()


@pytest.mark.parametrize("E,R,K", [(1, 16, 16), (2, 128, 256), (3, 144, 272), (1, 400, 128)])
def test_quantize_weight(zb, E, R, K):
    W = dev(np.stack([_rows(np.random.default_rng(e), R, K) for e in range(E)]))
    rb, cb = -(-R // 128), -(-K // 128)
    Q, S, QT, ST = e4(E, R, K), empty_f32(E, rb, cb), e4(E, K, R), empty_f32(E, cb, rb)
    zb.zb_fp8_quantize_weight(E, R, K, W, Q, S, QT, ST)
    Q2, S2, QT2, ST2 = e4(E, R, K), empty_f32(E, rb, cb), e4(E, K, R), empty_f32(E, cb, rb)
    zb.zb_fp8_quantize_weight(E, R, K, W, Q2, S2, None, None)
    zb.zb_fp8_quantize_weight(E, R, K, W, None, None, QT2, ST2)
    sync(zb)
    for e in range(E):
        q, s = om.quantize_weight(f64(W)[e])
        for Qx, Sx in ((Q, S), (Q2, S2)):
            assert np.array_equal(f64(Sx)[e], s) and np.array_equal(values(Qx)[e], q)
        for Qx, Sx in ((QT, ST), (QT2, ST2)):
            assert np.array_equal(f64(Sx)[e], s.T) and np.array_equal(values(Qx)[e], q.T)


CASES = [
    # counts (None: no offsets, that many rows), N, K, epilogue, act, bias, extra rows
    (1, 8, 16, "store", "erf", False, 0),
    (70, 136, 144, "store", "erf", True, 0),
    (300, 520, 1040, "gelu", "erf", True, 0),
    (257, 264, 384, "grad", "tanh", False, 0),
    ([0, 3, 129], 256, 128, "store", "erf", False, 4),
    ([16, 1, 0, 31, 33, 300], 200, 272, "gelu", "tanh", False, 0),
    ([130, 0, 0, 64, 257, 5], 392, 656, "grad", "erf", False, 9),
    ([600, 40, 513], 512, 512, "store", "erf", True, 0),
    # enough tiles for CTA pairs
    ([290, 1, 257, 0, 40, 513, 96, 33] * 2, 1288, 144, "grad", "erf", False, 7),
    ([290, 1, 257, 0, 40, 513, 96, 33] * 2, 1288, 272, "gelu", "erf", True, 0),
    (2500, 2056, 400, "store", "erf", True, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("scales", ["powers", "any"])
def test_matmul(zb, case, scales):
    counts, N, K, epi, act, bias, extra = CASES[case]
    rng = np.random.default_rng(case)
    dense = isinstance(counts, int)
    cl = [counts] if dense else counts
    E, M = len(cl), sum(cl) + extra
    off = np.concatenate([[0], np.cumsum(cl)])
    live = int(off[-1])
    kb, nb = -(-K // 128), -(-N // 128)
    X, W = dev(rng.normal(size=(M, K)) * np.exp2(rng.integers(-4, 4, size=(M, 1)))), dev(rng.normal(size=(E, K, N)) / np.sqrt(K))
    # N need not be a multiple of 16 for the product; the weight quantiser's rows and columns must
    Wp = torch.zeros(E, K, -(-N // 16) * 16, dtype=torch.bfloat16, device="cuda")
    Wp[:, :, :N] = W
    Xq, Xs = e4(M, K), empty_f32(M, kb)
    QT, ST = e4(E, Wp.shape[2], K), empty_f32(E, nb, kb)
    zb.zb_fp8_quantize_rows(M, K, X, Xq, Xs)
    zb.zb_fp8_quantize_weight(E, K, Wp.shape[2], Wp, None, None, QT, ST)
    sync(zb)
    Wq = QT.view(torch.uint8)[:, :N].contiguous().view(E4)
    if scales == "any":
        Xs = Xs * torch.rand_like(Xs)
        ST = ST * (0.5 + torch.rand_like(ST))
    Xs[live:] = NAN
    b = dev(rng.normal(size=(E, N))) if bias else None
    H = dev(rng.normal(size=(M, N)))
    o0, o1 = empty_bf16(M, N), empty_bf16(M, N)
    acts = {"erf": zb.ZB_ACT_GELU_ERF, "tanh": zb.ZB_ACT_GELU_TANH}
    epis = {"store": zb.ZB_FP8_STORE, "gelu": zb.ZB_FP8_GELU, "grad": zb.ZB_FP8_GELU_GRAD}
    g = zb.make_fp8_matmul(M, N, K, E, epis[epi], acts[act],
                           zb.ZB_FP8_SCALE_ANY if scales == "any" else zb.ZB_FP8_SCALE_POW2)
    zb.zb_fp8_matmul(g, None if dense else i32(off), Xq, Xs, Wq, ST, H if epi == "grad" else None, o0,
                     o1 if epi == "gelu" else None, bias=b)
    sync(zb)
    xv = values(Xq) * om.spread_scales(f64(Xs), M, K, 1)
    wv = np.stack([values(Wq)[e] * om.spread_scales(f64(ST)[e], N, K, 128) for e in range(E)])
    ref, mag = om.by_expert(off, xv, wv.transpose(0, 2, 1), f64(b) if bias else None)
    err = (K + kb) * 2.0 ** -23 * mag
    name = "gelu_" + act
    with np.errstate(invalid="ignore"):
        if epi == "grad":
            h = f64(H)
            gp = ref * om.gelu_prime(h, name)
            near(o0, gp, 2.0 ** -8 * np.abs(gp) + 1.2 * err + 1e-6 * (1 + np.abs(h)) * np.abs(ref))
        else:
            near(o0, ref, 2.0 ** -8 * np.abs(ref) + err)
        if epi == "gelu":
            ga = om.gelu(ref, name)
            near(o1, ga, 2.0 ** -8 * np.abs(ga) + 1.2 * err + 1e-6 * np.abs(ref))
    assert torch.isnan(o0[live:]).all()


def test_matmul_scale_of_nan_reaches_its_row_only(zb):
    M, N, K = 40, 136, 256
    X = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    X[7, 130] = float("inf")
    Xq, Xs, Q, S = e4(M, K), empty_f32(M, 2), e4(1, 144, K), empty_f32(1, 2, 2)
    zb.zb_fp8_quantize_rows(M, K, X, Xq, Xs)
    zb.zb_fp8_quantize_weight(1, 144, K, torch.ones(1, 144, K, dtype=torch.bfloat16, device="cuda"), Q, S, None, None)
    out = empty_bf16(M, N)
    zb.zb_fp8_matmul(zb.make_fp8_matmul(M, N, K), None, Xq, Xs, Q, S, None, out, None)
    sync(zb)
    o = f64(out)
    assert np.isnan(o[7]).all()
    assert (np.delete(o, 7, axis=0) == K).all()


def test_matmul_without_rows(zb):
    out = empty_bf16(4, 8)
    zb.zb_fp8_matmul(zb.make_fp8_matmul(0, 8, 16), None, None, None, None, None, None, None, None)
    W, S = e4(2, 8, 16), empty_f32(2, 1, 1)
    X, xs = e4(4, 16), empty_f32(4, 1)
    zb.zb_fp8_matmul(zb.make_fp8_matmul(4, 8, 16, experts=2), i32([0, 0, 0]), X, xs, W, S, None, out, None)
    zb.zb_fp8_quantize_rows(0, 16, None, None, None)
    sync(zb)
    assert torch.isnan(out).all()
