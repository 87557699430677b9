"""GPU parity of the mixture-of-experts operators against the fp64 oracle.

Each output is compared with the oracle computed from the exact tensors the
kernel read.  Element-wise bounds, derived from the arithmetic:

* a bf16 output of an fp32 sum of n products differs from the exact value v by
  at most half a bf16 step, 2^-8 |v| (8 significant bits), plus the sum's own
  error, at most n 2^-23 times the sum of the absolute products (2^-23 rather
  than 2^-24: tensor cores may truncate);
* GeLU and GeLU' add the library's approximation error, below 1e-6 in Phi
  (formula error 1.5e-7, fast exponential and reciprocal), times |x| or |dA|;
* fp32 outputs: the sum's error alone.
"""

import numpy as np
import pytest
import torch

from oracle import moe as om
from tests.gpu_util import empty_bf16, empty_f32, f64, have_gpu, sync

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def zb():
    if not have_gpu():
        pytest.skip("no CUDA device")
    from split_backward_gemms_gb300 import build as B
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


def dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype).cuda()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def near(got, ref, bound):
    got, ref = f64(got), np.asarray(ref)
    same = np.isnan(ref) & np.isnan(got) | (ref == got)
    bad = ~(np.abs(got - ref) <= bound) & ~same
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


# ------------------------------------------------------------------- router
def _logits(T, E, seed, masked=0.0, padded=()):
    rng = np.random.default_rng(seed)
    z = np.round(rng.normal(size=(T, E)) * 4) / 4  # steps of 1/4: many ties
    if masked:
        z[rng.random((T, E)) < masked] = -np.inf
    z[list(padded)] = -np.inf
    return z


def _route(zb, z, k, renorm, dtype):
    T, E = z.shape
    lg = dev(z, dtype)
    out = dict(gates=empty_f32(T, k), expert=i32(np.full((T, k), 77)), offsets=i32(np.full(E + 1, 77)),
               row_of=i32(np.full((T, k), 77)), token_of=i32(np.full(T * k, 77)))
    r = zb.make_router(T, E, k, zb.ZB_DT_BF16 if dtype == torch.bfloat16 else zb.ZB_DT_F32, renorm)
    n = zb.zb_moe_route_workspace_bytes(r)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    zb.zb_moe_route(r, lg, out["gates"], out["expert"], out["offsets"], out["row_of"], out["token_of"], ws, n)
    sync(zb)
    return r, lg, out


@pytest.mark.parametrize("T,E,k,renorm,dtype", [
    (1, 1, 1, False, torch.float32), (1, 8, 2, True, torch.float32), (5, 33, 3, False, torch.bfloat16),
    (17, 64, 6, True, torch.float32), (32, 256, 32, False, torch.bfloat16), (33, 256, 8, True, torch.float32),
    (127, 64, 6, True, torch.float32), (128, 256, 8, False, torch.float32), (129, 60, 4, True, torch.bfloat16),
    (300, 65, 32, False, torch.float32), (1000, 129, 8, True, torch.float32), (4867, 16, 2, False, torch.bfloat16),
    (20011, 40, 2, True, torch.float32)])
def test_route(zb, T, E, k, renorm, dtype):
    z = _logits(T, E, T + E, masked=0.2 if E > 1 else 0.0, padded=range(0, T, 7) if T > 1 else ())
    _, lg, out = _route(zb, z, k, renorm, dtype)
    gates, expert, offsets, row_of, token_of = om.route(f64(lg), k, renorm)
    for name, ref in (("expert", expert), ("offsets", offsets), ("row_of", row_of), ("token_of", token_of)):
        assert np.array_equal(out[name].cpu().numpy(), ref), name
    # exp to 2 ulp, a sum of E terms, one division
    near(out["gates"], gates, (E + 8) * 2.0 ** -23 * gates)


def test_route_infinities_and_nan(zb):
    z = np.array([[0.0, -0.0, -INF, 0.0],       # -0 ties with +0: lowest index first
                  [-INF] * 4,                   # nothing left
                  [NAN, 1.0, -INF, 2.0],        # NaN chosen last, gates NaN
                  [INF, 1.0, 0.0, -1.0],
                  [-3.4028235e38, -INF, -INF, -INF],   # the type's lowest value is a number
                  [-3.4028235e38, 3.0, NAN, -INF],
                  [-1e30, -1e30, 1e30, -INF]])
    for renorm in (False, True):
        _, lg, out = _route(zb, z, 3, renorm, torch.float32)
        gates, expert, offsets, row_of, token_of = om.route(f64(lg), 3, renorm)
        for name, ref in (("expert", expert), ("offsets", offsets), ("row_of", row_of), ("token_of", token_of)):
            assert np.array_equal(out[name].cpu().numpy(), ref), name
        near(out["gates"], gates, 16 * 2.0 ** -23 * np.nan_to_num(gates))


def test_route_no_tokens(zb):
    r = zb.make_router(0, 7, 2)
    off = i32(np.full(8, 5))
    ws = torch.empty(zb.zb_moe_route_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    zb.zb_moe_route(r, None, None, None, off, None, None, ws, ws.numel())
    zb.zb_moe_route_backward(r, None, None, None, None, None)
    zb.zb_moe_dispatch(0, 2, 64, None, None, None)
    zb.zb_moe_combine(0, 2, 64, None, None, None, None)
    zb.zb_moe_combine_backward(0, 2, 64, None, None, None, None, None, None)
    sync(zb)
    assert (off == 0).all()


@pytest.mark.parametrize("T,E,k,renorm,dtype", [
    (1, 1, 1, False, torch.float32), (3, 8, 2, True, torch.float32), (9, 40, 8, False, torch.bfloat16),
    (130, 100, 4, True, torch.bfloat16), (67, 256, 32, False, torch.float32)])
def test_route_backward(zb, T, E, k, renorm, dtype):
    z = _logits(T, E, 3 * T + E, masked=0.2 if E > 1 else 0.0, padded=[0] if T > 1 else ())
    r, lg, out = _route(zb, z, k, renorm, dtype)
    dg = dev(np.random.default_rng(5).normal(size=(T, k)), torch.float32)
    dz = torch.full((T, E), NAN, dtype=dtype, device="cuda")
    zb.zb_moe_route_backward(r, lg, out["expert"], out["gates"], dg, dz)
    sync(zb)
    ref = om.route_backward(f64(lg), out["expert"].cpu().numpy(), f64(dg), renorm)
    # a product of a gate (exact to E + 8 ulp) and a difference of sums of k products below sum |dg|
    size = np.abs(f64(dg)).sum(1, keepdims=True)
    step = 2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0.0
    near(dz, ref, step + (E + 2 * k + 16) * 2.0 ** -23 * size)


@pytest.mark.parametrize("E", [7, 40, 100, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_masked_logits_get_no_gradient(zb, E, dtype, renorm):
    """Logits of -inf get zeros whatever the rest of their row holds."""
    k = 3
    z = np.random.default_rng(E).normal(size=(7, E)) * 2
    z[:, 1::3] = -INF
    z[3, 0], z[4, 0] = NAN, INF
    z[5] = -INF
    r, lg, out = _route(zb, z, k, renorm, dtype)
    dgn = np.random.default_rng(5).normal(size=(7, k))
    dgn[1, 1], dgn[2, 0], dgn[5, 0] = NAN, INF, NAN
    dg = dev(dgn, torch.float32)
    dz = torch.full((7, E), NAN, dtype=dtype, device="cuda")
    zb.zb_moe_route_backward(r, lg, out["expert"], out["gates"], dg, dz)
    sync(zb)
    got, masked = f64(dz), np.isneginf(f64(lg))
    assert (got[masked] == 0).all()
    chosen = np.zeros((7, E), bool)
    for t, e in np.argwhere(out["expert"].cpu().numpy() >= 0):
        chosen[t, int(out["expert"][t, e])] = True
    # what is not finite reaches every logit that has a weight
    for t in (1, 2, 3, 4):
        assert not np.isfinite(got[t][chosen[t] if renorm else ~masked[t]]).any()
    ref = om.route_backward(f64(lg)[[0, 6]], out["expert"].cpu().numpy()[[0, 6]], dgn.astype(np.float32)[[0, 6]], renorm)
    step = 2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0.0
    near(dz[[0, 6]], ref, step + (E + 2 * k + 16) * 2.0 ** -23 * np.abs(dgn[[0, 6]]).sum(1, keepdims=True))


# --------------------------------------------------------------------- rows
@pytest.mark.parametrize("T,E,k,w", [(1, 1, 1, 8), (3, 4, 2, 1032), (65, 8, 3, 520), (130, 32, 8, 2056),
                                     (257, 16, 2, 4104), (40, 64, 32, 136)])
def test_rows(zb, T, E, k, w):
    rng = np.random.default_rng(T + w)
    z = _logits(T, E, T, padded=[0] if T > 1 else ())
    gates, _, offsets, row_of, token_of = om.route(z, k, True)
    live, R = int(offsets[-1]), T * k
    X, Yp, dY = dev(rng.normal(size=(T, w))), dev(rng.normal(size=(R, w))), dev(rng.normal(size=(T, w)))
    Yp[live:] = NAN  # rows nobody owns
    ro, g = i32(row_of), dev(gates, torch.float32)
    Xp = empty_bf16(R, w)
    zb.zb_moe_dispatch(T, k, w, X, ro, Xp)
    Y, Y1 = empty_bf16(T, w), empty_bf16(T, w)
    zb.zb_moe_combine(T, k, w, Yp, ro, g, Y)
    zb.zb_moe_combine(T, k, w, Yp, ro, None, Y1)
    dYp, dg = empty_bf16(R, w), empty_f32(T, k)
    zb.zb_moe_combine_backward(T, k, w, dY, Yp, ro, g, dYp, dg)
    sync(zb)
    assert np.array_equal(f64(Xp)[:live], f64(X)[token_of[:live]])
    assert torch.isnan(Xp[live:]).all() and torch.isnan(dYp[live:]).all()
    for got, gg in ((Y, f64(g)), (Y1, None)):
        ref = om.combine(f64(Yp), row_of, gg)
        mag = om.combine(np.abs(f64(Yp)), row_of, gg)
        near(got, ref, 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * mag)
    rY, rg = om.combine_backward(f64(dY), f64(Yp), row_of, f64(g))
    near(dYp, rY, 2.0 ** -8 * np.abs(rY))
    _, mag = om.combine_backward(np.abs(f64(dY)), np.abs(f64(Yp)), row_of, f64(g))
    near(dg, rg, w * 2.0 ** -23 * mag)


# ------------------------------------------------------------------ experts
CASES = [
    # counts, h, f, act, bias, rows past the last expert's
    ([1], 8, 8, "erf", False, 0),
    ([0, 0, 3], 72, 200, "tanh", True, 5),
    ([16, 1, 0, 31, 33], 64, 128, "erf", True, 0),
    ([129, 0, 127, 257, 2], 136, 264, "erf", False, 40),
    ([300, 513, 64], 256, 512, "erf", True, 0),
    ([700, 20, 0, 0, 1100], 264, 1032, "tanh", False, 3),
    ([5, 17, 8, 0, 2, 40] * 10, 128, 384, "erf", False, 0),
    # enough tiles for CTA pairs on either side
    ([290, 1, 257, 0, 40, 513, 96, 33] * 2, 136, 1288, "erf", True, 7),
    ([290, 1, 257, 0, 40, 513, 96, 33] * 2, 1288, 136, "tanh", False, 0),
    ([200, 90], 320, 136, "none", True, 1),
    ([3, 0, 70], 40, 72, "none", False, 0),
    # few rows an expert on average: tiles of 32 rows, 64 and 128 columns wide; some experts have more
    ([100, 1, 0, 2, 1, 1, 1, 33], 264, 1032, "erf", True, 3),
    ([7, 1, 0, 2, 33, 1, 1, 1], 136, 1288, "tanh", True, 0),
    ([1], 1352, 72, "none", True, 0),
    # long experts: bias gradients summed in parts
    ([1100, 3, 0, 2500], 72, 136, "erf", True, 1),
    ([5001], 8, 72, "none", True, 0),
    # many experts, nearly all with a partial last block, narrow matrices on CTA pairs
    ([148, 286, 0, 138, 60, 165, 78, 12, 81, 57, 307, 23, 277, 37, 14, 472] * 4, 48, 48, "erf", False, 2),
    ([17, 3, 7, 0, 30, 0, 6, 15, 2, 64, 5, 1, 128] * 10, 264, 136, "tanh", True, 0),
]


def _setup(zb, counts, h, f, act, bias, extra, seed=0):
    rng = np.random.default_rng(seed)
    E, R = len(counts), sum(counts) + extra
    off = np.concatenate([[0], np.cumsum(counts)])
    acts = {"erf": zb.ZB_ACT_GELU_ERF, "tanh": zb.ZB_ACT_GELU_TANH, "none": zb.ZB_ACT_NONE}
    m = zb.make_moe(R, h, f, E, acts[act], bias)
    s = dict(W1=dev(rng.normal(size=(E, h, f)) / np.sqrt(h)), W2=dev(rng.normal(size=(E, f, h)) / np.sqrt(f)),
             b1=dev(rng.normal(size=(E, f))), b2=dev(rng.normal(size=(E, h))),
             X=dev(rng.normal(size=(R, h))), dY=dev(rng.normal(size=(R, f if act == "none" else h))))
    live = int(off[-1])
    s["X"][live:] = NAN  # what is past the last expert's rows is not read
    s["dY"][live:] = NAN
    return m, off, i32(off), s, live


@pytest.mark.parametrize("case", range(len(CASES)))
def test_experts(zb, case):
    counts, h, f, act, bias, extra = CASES[case]
    m, off, offd, s, live = _setup(zb, counts, h, f, act, bias, extra, case)
    E, R = len(counts), sum(counts) + extra
    mlp = act != "none"
    b1, b2 = (s["b1"], s["b2"]) if bias else (None, None)
    n_out = h if mlp else f
    H, A, Y = empty_bf16(R, f), empty_bf16(R, f), empty_bf16(R, n_out)
    dH, dX = empty_bf16(R, f), empty_bf16(R, h)
    zb.zb_moe_forward(m, offd, s["X"], s["W1"], s["W2"], b1, b2, H, A, Y)
    zb.zb_moe_backward_input(m, offd, s["dY"], s["W1"], s["W2"], H, dH, dX)
    sync(zb)
    W1, W2 = f64(s["W1"]), f64(s["W2"])
    name = "gelu_" + act
    lin, mag = om.by_expert(off, f64(s["X"]), W1, f64(b1) if bias else None)
    err = h * 2.0 ** -23 * mag
    if not mlp:
        near(Y, lin, 2.0 ** -8 * np.abs(lin) + err)
        ref, mag = om.by_expert(off, f64(s["dY"]), W1.transpose(0, 2, 1))
        near(dX, ref, 2.0 ** -8 * np.abs(ref) + f * 2.0 ** -23 * mag)
        assert torch.isnan(Y[live:]).all() and torch.isnan(dX[live:]).all()
        return
    near(H, lin, 2.0 ** -8 * np.abs(lin) + err)
    with np.errstate(invalid="ignore"):
        ga = om.gelu(lin, name)
        # |GeLU'| <= 1.13; the form's own error 1e-6 |x|
        near(A, ga, 2.0 ** -8 * np.abs(ga) + 1.2 * err + 1e-6 * np.abs(lin))
        ref, mag = om.by_expert(off, f64(A), W2, f64(b2) if bias else None)
        near(Y, ref, 2.0 ** -8 * np.abs(ref) + f * 2.0 ** -23 * mag)
        dA, mag = om.by_expert(off, f64(s["dY"]), W2.transpose(0, 2, 1))
        gp = om.gelu_prime(f64(H), name)
        ref = dA * gp
        # |GeLU'| <= 1.13; its form's own error 1e-6 (1 + |x|)
        near(dH, ref, 2.0 ** -8 * np.abs(ref) + 1.2 * h * 2.0 ** -23 * mag + 1e-6 * (1 + np.abs(f64(H))) * np.abs(dA))
        ref, mag = om.by_expert(off, f64(dH), W1.transpose(0, 2, 1))
        near(dX, ref, 2.0 ** -8 * np.abs(ref) + f * 2.0 ** -23 * mag)
    for t in (H, A, Y, dH, dX):
        assert torch.isnan(t[live:]).all()


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_experts_weight_gradient(zb, case, accumulate):
    counts, h, f, act, bias, extra = CASES[case]
    m, off, offd, s, live = _setup(zb, counts, h, f, act, bias, extra, case + 50)
    E, R = len(counts), sum(counts) + extra
    mlp = act != "none"
    rng = np.random.default_rng(case)
    A, dH = dev(rng.normal(size=(R, f))), dev(rng.normal(size=(R, f)))
    A[live:] = NAN
    dH[live:] = NAN
    start = [dev(rng.normal(size=sh), torch.float32) for sh in ((E, h, f), (E, f, h), (E, f), (E, h))]
    got = [t.clone() if accumulate else torch.full_like(t, NAN) for t in start]
    n = zb.zb_moe_workspace_bytes(m)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    zb.zb_moe_backward_weight(m, offd, s["X"], A, dH, s["dY"], got[0], got[1], got[2], got[3], accumulate, ws, n)
    sync(zb)
    g1 = f64(dH) if mlp else f64(s["dY"])
    X, Af, dY = f64(s["X"]), f64(A), f64(s["dY"])
    pairs = [(got[0], start[0], X, g1)] + ([(got[1], start[1], Af, dY)] if mlp else [])
    for t, t0, a, b in pairs:
        for e, lo, hi in om.spans(off):
            ref = a[lo:hi].T @ b[lo:hi] + (f64(t0)[e] if accumulate else 0.0)
            mag = np.abs(a[lo:hi]).T @ np.abs(b[lo:hi]) + (np.abs(f64(t0)[e]) if accumulate else 0.0)
            near(t[e], ref, (hi - lo + 1) * 2.0 ** -23 * mag)
    if bias:
        sums = [(got[2], start[2], g1)] + ([(got[3], start[3], dY)] if mlp else [])
        for t, t0, b in sums:
            for e, lo, hi in om.spans(off):
                ref = b[lo:hi].sum(0) + (f64(t0)[e] if accumulate else 0.0)
                mag = np.abs(b[lo:hi]).sum(0) + (np.abs(f64(t0)[e]) if accumulate else 0.0)
                near(t[e], ref, (hi - lo + 1) * 2.0 ** -23 * mag)


@pytest.mark.parametrize("counts,h,f", [([2500], 264, 520), ([5001, 64, 700], 136, 256)])
def test_experts_weight_gradient_of_long_experts(zb, counts, h, f):
    """W's sums are cut into accumulators of 512 rows.  Each of an accumulator's
    512 / 16 adds cuts off half a step of the partial sum on average, 0.72 2^-24
    of its size; partial sums of independent terms grow as the root of their
    number, so the cuts come to 0.72 2^-24 (2/3) (512 / 16) of the result, and
    the s accumulators' own fp32 sum adds at most 2^-24 sqrt(s).  (One accumulator
    over 2500 rows would be 2.6e-6 off.)"""
    m, off, offd, s, _ = _setup(zb, counts, h, f, "erf", False, 0, 31)
    R, E = sum(counts), len(counts)
    rng = np.random.default_rng(32)
    A, dH = dev(rng.normal(size=(R, f))), dev(rng.normal(size=(R, f)))
    dW1, dW2 = empty_f32(E, h, f), empty_f32(E, f, h)
    n = zb.zb_moe_workspace_bytes(m)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    zb.zb_moe_backward_weight(m, offd, s["X"], A, dH, s["dY"], dW1, dW2, None, None, 0, ws, n)
    sync(zb)
    for e, lo, hi in om.spans(off):
        tol = 2.0 ** -24 * (0.72 * 2 / 3 * 32 + (-(-(hi - lo) // 512)) ** 0.5)
        for t, a, b in ((dW1, s["X"], dH), (dW2, A, s["dY"])):
            ref = f64(a)[lo:hi].T @ f64(b)[lo:hi]
            assert np.linalg.norm(f64(t[e]) - ref) < tol * np.linalg.norm(ref)


def test_offsets_at_any_word(zb):
    """Offsets of several microbatches in one tensor: the second one's are read
    from a 4-byte boundary."""
    counts, h, f = [37, 0, 90, 21], 144, 208
    m, off, offd, s, _ = _setup(zb, counts, h, f, "erf", True, 0, 12)
    R, E = sum(counts), len(counts)
    both = i32(np.stack([np.zeros(E + 1), off]))  # rows of 5 words
    assert both[1].data_ptr() % 16
    runs = []
    for o in (offd, both[1]):
        H, A, Y, dH, dX = empty_bf16(R, f), empty_bf16(R, f), empty_bf16(R, h), empty_bf16(R, f), empty_bf16(R, h)
        grads = [empty_f32(E, h, f), empty_f32(E, f, h), empty_f32(E, f), empty_f32(E, h)]
        n = zb.zb_moe_workspace_bytes(m)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        zb.zb_moe_forward(m, o, s["X"], s["W1"], s["W2"], s["b1"], s["b2"], H, A, Y)
        zb.zb_moe_backward_input(m, o, s["dY"], s["W1"], s["W2"], H, dH, dX)
        zb.zb_moe_backward_weight(m, o, s["X"], A, dH, s["dY"], *grads, 0, ws, n)
        Xq, Xs = torch.zeros(R, h, dtype=torch.uint8, device="cuda"), empty_f32(R, 2)
        Wq, Ws = torch.zeros(E, f, h, dtype=torch.uint8, device="cuda"), empty_f32(E, 2, 2)
        Z = empty_bf16(R, f)
        zb.zb_fp8_quantize_rows(R, h, s["X"], Xq, Xs)
        zb.zb_fp8_quantize_weight(E, h, f, s["W1"], None, None, Wq, Ws)
        zb.zb_fp8_matmul(zb.make_fp8_matmul(R, f, h, E), o, Xq, Xs, Wq, Ws, None, Z, None)
        sync(zb)
        runs.append([H, A, Y, dH, dX, Z] + grads)
    for a, b in zip(*runs):
        assert torch.equal(a, b) and not torch.isnan(a).any()


def test_experts_do_not_touch_each_other(zb):
    """NaN and infinities in one expert's weights or rows stay in its own results."""
    counts, h, f = [37, 0, 90, 21], 136, 200
    m, off, offd, s, _ = _setup(zb, counts, h, f, "erf", False, 0, 9)
    R = sum(counts)
    E = len(counts)

    def passes():
        o = dict(H=empty_bf16(R, f), A=empty_bf16(R, f), Y=empty_bf16(R, h), dH=empty_bf16(R, f), dX=empty_bf16(R, h),
                 dW1=empty_f32(E, h, f), dW2=empty_f32(E, f, h))
        zb.zb_moe_forward(m, offd, s["X"], s["W1"], s["W2"], None, None, o["H"], o["A"], o["Y"])
        zb.zb_moe_backward_input(m, offd, s["dY"], s["W1"], s["W2"], o["H"], o["dH"], o["dX"])
        n = zb.zb_moe_workspace_bytes(m)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        zb.zb_moe_backward_weight(m, offd, s["X"], o["A"], o["dH"], s["dY"], o["dW1"], o["dW2"], None, None, 0, ws, n)
        sync(zb)
        return o

    clean = passes()
    for t in ("W1", "W2"):
        s[t][1] = INF      # an expert without rows
        s[t][2] = NAN
    s["X"][127:] = INF     # expert 3's rows
    s["dY"][127:] = NAN
    dirty = passes()
    for e in (0,):
        a, b = int(off[e]), int(off[e + 1])
        for t in ("H", "A", "Y", "dH", "dX"):
            assert torch.equal(clean[t][a:b], dirty[t][a:b]), t
        for t in ("dW1", "dW2"):
            assert torch.equal(clean[t][e], dirty[t][e]), t
    for t in ("dW1", "dW2"):
        assert (dirty[t][1] == 0).all(), t
    assert torch.isnan(dirty["Y"][37:127]).all()
    # dW1 of the expert with NaN weights: its dH is NaN; dW2 of it reads A = NaN
    assert torch.isnan(dirty["dW1"][2]).all() and torch.isnan(dirty["dW2"][3]).all()


def test_experts_on_another_stream_repeat_bits(zb):
    counts, h, f = [100, 260, 0, 33], 264, 392
    m, off, offd, s, _ = _setup(zb, counts, h, f, "erf", True, 0, 4)
    R, E = sum(counts), len(counts)
    runs = []
    torch.cuda.synchronize()
    for _ in range(2):
        st = torch.cuda.Stream()
        H, A, Y, dH, dX = empty_bf16(R, f), empty_bf16(R, f), empty_bf16(R, h), empty_bf16(R, f), empty_bf16(R, h)
        dW1, dW2, db1, db2 = empty_f32(E, h, f), empty_f32(E, f, h), empty_f32(E, f), empty_f32(E, h)
        n = zb.zb_moe_workspace_bytes(m)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        zb.zb_moe_forward(m, offd, s["X"], s["W1"], s["W2"], s["b1"], s["b2"], H, A, Y, stream=st)
        zb.zb_moe_backward_input(m, offd, s["dY"], s["W1"], s["W2"], H, dH, dX, stream=st)
        zb.zb_moe_backward_weight(m, offd, s["X"], A, dH, s["dY"], dW1, dW2, db1, db2, 0, ws, n, stream=st)
        st.synchronize()
        sync(zb)
        runs.append((H, A, Y, dH, dX, dW1, dW2, db1, db2))
    for a, b in zip(*runs):
        assert torch.equal(a, b) and not torch.isnan(a).any()


def test_one_expert_matches_the_block(zb):
    """E = 1 is the dense block: the same passes, up to the order of sums."""
    M, h, f = 333, 256, 1024
    m, off, offd, s, _ = _setup(zb, [M], h, f, "erf", False, 0, 6)
    blk = zb.make_block(M, h, f)
    H, A, Y, dH, dX = empty_bf16(M, f), empty_bf16(M, f), empty_bf16(M, h), empty_bf16(M, f), empty_bf16(M, h)
    Hb, Ab, Yb, dHb, dXb = (torch.empty_like(t) for t in (H, A, Y, dH, dX))
    zb.zb_moe_forward(m, offd, s["X"], s["W1"], s["W2"], None, None, H, A, Y)
    zb.zb_moe_backward_input(m, offd, s["dY"], s["W1"], s["W2"], H, dH, dX)
    zb.zb_forward(blk, s["X"], s["W1"], s["W2"], None, None, Hb, Ab, Yb)
    zb.zb_backward_input(blk, s["dY"], s["W1"], s["W2"], Hb, dHb, dXb)
    sync(zb)
    for a, b in ((H, Hb), (A, Ab), (Y, Yb), (dH, dHb), (dX, dXb)):
        d = (a.double() - b.double()).norm() / b.double().norm()
        assert d < 5e-3, float(d)
