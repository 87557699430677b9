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


# Scales that differ from block to block, and enough blocks of K or tiles to take
# the hand-over of scales (16 blocks of K a batch, two batches in shared memory,
# eight groups of four blocks in tensor memory) more than once round.
LONG = [
    # counts (None: no offsets), N, K, epilogue
    (70, 136, 2064, "store"),                # 17 blocks: a second, partial batch
    (70, 136, 2304, "grad"),
    ([5, 0, 129, 40], 264, 4096, "gelu"),    # 32: two whole batches, scales in 16-byte loads
    (200, 264, 4224, "store"),               # 33: a slot used again within a tile, a ninth group
    ([3, 140], 136, 4224, "grad"),
    (130, 136, 4608, "store"),               # 36, in 16-byte loads
    (300, 264, 6160, "grad"),                # 49: four batches
    ([9, 31, 3, 0, 70, 1, 17, 2] * 11, 520, 2064, "store"),      # CTA pairs, three tiles a pair and more
    ([9, 31, 3, 0, 70, 1, 17, 2] * 11, 520, 2064, "grad"),
    ([2, 5, 0, 3, 1, 7, 4, 2] * 32, 776, 144, "store"),          # pairs, eleven tiles each: groups go round
    ([2, 5, 0, 3, 1, 7, 4, 2] * 32, 776, 144, "gelu"),
    ([257, 255, 256] * 25, 136, 400, "store"),                   # single CTAs, some with a second tile
    ([257, 255, 256] * 25, 136, 2064, "grad"),
]


def _steps(rng, rows, cols, rb, lo, hi):
    """2^lo .. 2^hi for each block of rb x 128."""
    e = rng.integers(lo, hi + 1, size=(-(-rows // rb), -(-cols // 128)))
    return np.exp2(np.repeat(np.repeat(e, rb, axis=0), 128, axis=1)[:rows, :cols].astype(np.float64))


@pytest.mark.parametrize("scales", ["powers", "any"])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_matmul_of_many_blocks(zb, case, scales):
    counts, N, K, epi = LONG[case]
    rng = np.random.default_rng(100 + case)
    dense = isinstance(counts, int)
    cl = [counts] if dense else counts
    E, M = len(cl), sum(cl)
    off = np.concatenate([[0], np.cumsum(cl)])
    kb, nb, Np = -(-K // 128), -(-N // 128), -(-N // 16) * 16
    Xq, Xs = e4(M, K), empty_f32(M, kb)
    zb.zb_fp8_quantize_rows(M, K, dev(rng.normal(size=(M, K)) * _steps(rng, M, K, 1, -6, 6)), Xq, Xs)
    QT, ST = e4(E, Np, K), empty_f32(E, nb, kb)
    W = np.zeros((E, K, Np), np.float32)
    for e in range(E):
        W[e, :, :N] = rng.standard_normal((K, N), dtype=np.float32) * _steps(rng, K, N, 128, -6, 6)
    zb.zb_fp8_quantize_weight(E, K, Np, dev(W), None, None, QT, ST)
    del W
    sync(zb)
    Wq = QT.view(torch.uint8)[:, :N].contiguous().view(E4)
    if scales == "any":
        Xs = Xs * (0.5 + torch.rand_like(Xs))
        ST = ST * (0.5 + torch.rand_like(ST))
    H = dev(rng.normal(size=(M, N)))
    o0, o1 = empty_bf16(M, N), empty_bf16(M, N)
    g = zb.make_fp8_matmul(M, N, K, E, dict(store=zb.ZB_FP8_STORE, gelu=zb.ZB_FP8_GELU, grad=zb.ZB_FP8_GELU_GRAD)[epi],
                           zb.ZB_ACT_GELU_ERF, zb.ZB_FP8_SCALE_ANY if scales == "any" else zb.ZB_FP8_SCALE_POW2)
    zb.zb_fp8_matmul(g, None if dense else i32(off), Xq, Xs, Wq, ST, H if epi == "grad" else None, o0,
                     o1 if epi == "gelu" else None)
    sync(zb)
    xv = values(Xq) * om.spread_scales(f64(Xs), M, K, 1)
    ref, mag = np.zeros((M, N)), np.zeros((M, N))
    for e, a, b in om.spans(off):
        if b > a:
            wv = (values(Wq[e]) * om.spread_scales(f64(ST[e]), N, K, 128)).T
            ref[a:b], mag[a:b] = xv[a:b] @ wv, np.abs(xv[a:b]) @ np.abs(wv)
    err = (K + kb) * 2.0 ** -23 * mag
    if epi == "grad":
        h = f64(H)
        gp = ref * om.gelu_prime(h, "gelu_erf")
        near(o0, gp, 2.0 ** -8 * np.abs(gp) + 1.2 * err + 1e-6 * (1 + np.abs(h)) * np.abs(ref))
    else:
        near(o0, ref, 2.0 ** -8 * np.abs(ref) + err)
    if epi == "gelu":
        ga = om.gelu(ref, "gelu_erf")
        near(o1, ga, 2.0 ** -8 * np.abs(ga) + 1.2 * err + 1e-6 * np.abs(ref))


@pytest.mark.parametrize("scales", ["powers", "any"])
@pytest.mark.parametrize("M,N,K", [(70, 136, 400), (300, 2056, 400)])
def test_matmul_of_extreme_scales(zb, M, N, K, scales):
    """Blocks whose scales lie near either end of their range, the products in
    range: rows of 2^-126 (subnormal values) to 2^100 against weights of the
    inverse, another exponent for every block of K."""
    rng = np.random.default_rng(M)
    kb, nb, Np = -(-K // 128), -(-N // 128), -(-N // 16) * 16
    ex = np.array([-128, 100, -60, 3])[:kb]  # of the values; scales are 2^-126 and about 2^-6 of them
    of_k = np.exp2(np.repeat(ex, 128)[:K].astype(np.float64))
    X = rng.normal(size=(M, K)) * of_k
    W = np.zeros((1, K, Np))
    W[0, :, :N] = rng.normal(size=(K, N)) / of_k[:, None] * np.where(np.repeat(ex, 128)[:K, None] < -100, 2.0 ** -4, 1.0)
    Xq, Xs, QT, ST = e4(M, K), empty_f32(M, kb), e4(1, Np, K), empty_f32(1, nb, kb)
    zb.zb_fp8_quantize_rows(M, K, dev(X), Xq, Xs)
    zb.zb_fp8_quantize_weight(1, K, Np, dev(W), None, None, QT, ST)
    sync(zb)
    assert (f64(Xs)[:, 0] == 2.0 ** -126).all() and f64(Xs)[:, 1].min() > 2.0 ** 90
    Wq = QT.view(torch.uint8)[:, :N].contiguous().view(E4)
    if scales == "any":
        Xs = Xs * (1.0 + torch.rand_like(Xs))
    out = empty_bf16(M, N)
    zb.zb_fp8_matmul(zb.make_fp8_matmul(M, N, K, scales=zb.ZB_FP8_SCALE_ANY if scales == "any" else zb.ZB_FP8_SCALE_POW2),
                     None, Xq, Xs, Wq, ST, None, out, None)
    sync(zb)
    xv, wv = values(Xq) * om.spread_scales(f64(Xs), M, K, 1), values(Wq[0]) * om.spread_scales(f64(ST[0]), N, K, 128)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert (np.abs(xv[:, :128]) @ np.abs(wv[:, :128]).T).min() > 0.0  # the subnormal block counts
    near(out, ref, 2.0 ** -8 * np.abs(ref) + (K + kb) * 2.0 ** -23 * mag)


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
