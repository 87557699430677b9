"""GPU parity of the linear maps, layer norm and embedding against the fp64 oracle.

Each output is compared with the oracle computed from the exact tensors the
kernel read.  Element-wise bounds, derived from the arithmetic (e = 2^-24, half
an fp32 step; a bf16 output adds half a step of its own, 2^-8 |v|):

* linear: a sum of K products is off by at most K 2^-23 times the sum of the
  absolute products (2^-23 rather than 2^-24: tensor cores may truncate); bias
  and residual add two roundings; GeLU and GeLU' add the library's
  approximation error, below 1e-6 in Phi, times |x| or |D|, and pass the sum's
  error on with a slope of at most 1.13;
* norm: a row's sums have at most 64 + 5 + 16 roundings in a chain (values of a
  lane, shuffles, warps), a column's rows / 256 + 16 (values of a thread,
  shuffles, warps, blocks);
* embedding: a run's sum has at most 32 roundings in a piece and one for each of
  its pieces.
"""

import numpy as np
import pytest
import torch

from oracle import around as oa
from tests.gpu_util import empty_bf16, empty_f32, f64, have_gpu, sync

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
E = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def zb():
    if not have_gpu():
        pytest.skip("no CUDA device")
    from split_backward_gemms_gb300 import build as B
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


def dev(a, dtype=BF16):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype).cuda()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def near(got, ref, bound):
    got, ref = f64(got), np.asarray(ref)
    same = np.isnan(ref) & np.isnan(got) | (ref == got)
    bad = ~(np.abs(got - ref) <= bound) & ~same
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def bits(t):
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32)


def step(dtype):
    """Half a step of the type, relative."""
    return 2.0 ** -8 if dtype == BF16 else E


# ------------------------------------------------------------------- linear
def wide(a, gap, fill, dtype=BF16):
    """`a` as a slice of a buffer with `gap` more columns, which hold `fill`."""
    big = torch.full((a.shape[0], a.shape[1] + gap), fill, dtype=dtype, device="cuda")
    big[:, :a.shape[1]] = dev(a, dtype)
    return big, big[:, :a.shape[1]]


class Linear:
    def __init__(self, zb, M, N, K, form="store", transposed=False, dtype=BF16, bias=True, residual=True, save=True,
                 gap=0, tanh=False, seed=0):
        rng = np.random.default_rng(seed + M + 7 * N + 13 * K)
        self.zb, self.form, self.transposed, self.tanh, self.dtype = zb, form, transposed, tanh, dtype
        self.N, self.gap = N, gap
        _, self.X = wide(rng.normal(size=(M, K)), gap, NAN)
        _, self.W = wide(rng.normal(size=(N, K) if transposed else (K, N)) / np.sqrt(K), gap, NAN)
        self.bias = dev(rng.normal(size=N)) if bias and form != "grad" else None
        self.R = wide(rng.normal(size=(M, N)), gap, NAN, dtype)[1] if residual else None
        self.H = wide(rng.normal(size=(M, N)) * 2, gap, NAN)[1] if form == "grad" else None
        self.big, self.out = wide(np.zeros((M, N)), gap, 77.0, dtype)
        self.kept_big, self.kept = wide(np.zeros((M, N)), gap, 77.0) if form == "gelu" and save else (None, None)
        self.out.fill_(NAN)
        self.desc = zb.make_linear(
            M, N, K, transposed=transposed,
            epilogue={"store": zb.ZB_LINEAR_STORE, "gelu": zb.ZB_LINEAR_GELU, "grad": zb.ZB_LINEAR_GELU_GRAD}[form],
            act=zb.ZB_ACT_GELU_TANH if tanh else zb.ZB_ACT_GELU_ERF,
            dtype=zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32, ldx=K + gap,
            ldw=(K if transposed else N) + gap, ldr=N + gap, ldh=N + gap, ldo=N + gap)

    def run(self, stream=None):
        o0, o1 = (self.kept, self.out) if self.form == "gelu" else (self.out, None)
        self.zb.zb_linear_product(self.desc, self.X, self.W, self.bias, self.R, self.H, o0, o1, stream=stream)
        return self

    def check(self, R=None):
        sync(self.zb)
        X, W = f64(self.X), f64(self.W)
        bias = None if self.bias is None else f64(self.bias)
        H = None if self.H is None else f64(self.H)
        R = R if R is not None else None if self.R is None else f64(self.R)
        ref, D = oa.linear(X, W, self.transposed, self.form, bias, R, H, self.tanh)
        terms = np.abs(X) @ np.abs(W.T if self.transposed else W) + (0.0 if bias is None else np.abs(bias))
        off = (X.shape[1] + 2) * 2.0 ** -23 * terms
        if self.kept is not None:
            near(self.kept, D, off + 2.0 ** -8 * (np.abs(D) + off))
        if self.form != "store":
            # GeLU(D), or D GeLU'(H) with |GeLU'| <= 1.13
            off = 1.13 * off + 3e-6 * np.abs(D) * (1.0 if H is None else 1.0 + np.abs(H))
        if R is not None:
            off = off + 2 * E * (np.abs(ref) + np.abs(R))
        near(self.out, ref, off + step(self.dtype) * (np.abs(ref) + off))
        if self.gap:
            assert (self.big[:, self.N:] == 77.0).all()
            assert self.kept_big is None or (self.kept_big[:, self.N:] == 77.0).all()


SHAPES = [(1, 8, 8), (1, 64, 256), (3, 8, 16), (7, 136, 4096), (16, 1024, 4096), (17, 136, 200), (32, 2048, 64),
          (33, 264, 1032), (64, 1024, 1024), (65, 512, 2048), (127, 72, 520), (128, 256, 64), (129, 264, 72),
          (200, 520, 1032), (256, 4096, 1024), (300, 1024, 2056), (512, 1024, 1024), (1000, 2056, 520),
          (2049, 2048, 512), (4096, 1032, 264)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("form", ["store", "gelu", "grad"])
def test_linear(zb, M, N, K, form):
    k = SHAPES.index((M, N, K))
    Linear(zb, M, N, K, form, transposed=form == "grad" or k % 2 == 1, gap=(0, 8, 72)[k % 3], save=k % 4 < 2,
           tanh=k % 5 == 4, bias=k % 7 != 3).run().check()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_other_way(zb, M, N, K):
    """The other operand order, without residual or without bias."""
    k = SHAPES.index((M, N, K))
    Linear(zb, M, N, K, "store", transposed=k % 2 == 0, residual=k % 2 == 0, bias=k % 2 == 1).run().check()
    Linear(zb, M, N, K, "gelu", transposed=k % 2 == 0, residual=False, save=k % 4 >= 2, gap=8).run().check()
    Linear(zb, M, N, K, "grad", transposed=False, residual=k % 2 == 1, tanh=True).run().check()


@pytest.mark.parametrize("M,N,K", SHAPES + [(16, 256, 16384), (300, 512, 6144), (1100, 2048, 3000)])
@pytest.mark.parametrize("transposed", [False, True])
def test_linear_fp32(zb, M, N, K, transposed):
    c = Linear(zb, M, N, K, transposed=transposed, dtype=F32, gap=16 if K % 16 else 0, residual=M != 33,
               bias=M != 64).run()
    c.check()
    # fp32 sums: a random walk of K roundings, not K of them one way
    ref, _ = oa.linear(f64(c.X), f64(c.W), transposed, "store", None if c.bias is None else f64(c.bias),
                       None if c.R is None else f64(c.R))
    assert np.linalg.norm(f64(c.out) - ref) <= 1e-6 * np.linalg.norm(ref)


# tiles of 256, 224, 192, 160 and 128 columns where W lies along K; more column
# tiles than SMs; problems on either side of the rule between the two kernels
TILINGS = [(2100, 2056, 136), (2304, 1640, 200), (4096, 2400, 72), (3300, 1608, 72), (1500, 4008, 72), (700, 1000, 72),
           (20, 20488, 136), (40, 19448, 72), (40, 20488, 72), (65, 4104, 2048), (65, 4872, 2040), (130, 4104, 4096)]


@pytest.mark.parametrize("M,N,K", TILINGS)
@pytest.mark.parametrize("transposed", [False, True])
def test_linear_tilings(zb, M, N, K, transposed):
    gap = 8 * (N % 3)
    Linear(zb, M, N, K, "grad", transposed=transposed, gap=gap).run().check()
    Linear(zb, M, N, K, "gelu", transposed=transposed, gap=gap, save=transposed).run().check()
    Linear(zb, M, N, K, transposed=transposed, dtype=F32, gap=gap).run().check()


@pytest.mark.parametrize("M,N,K,dtype", [(5, 64, 512, BF16), (300, 1032, 520, BF16), (2048, 2048, 256, BF16),
                                         (40, 1024, 2048, F32), (2048, 1032, 256, F32)])
def test_linear_in_place(zb, M, N, K, dtype):
    """The output is the residual itself."""
    c = Linear(zb, M, N, K, dtype=dtype)
    R = f64(c.R)
    c.out = c.R
    c.run().check(R)


@pytest.mark.parametrize("M,N,K", [(9, 72, 136), (130, 520, 264), (2100, 2048, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_infinities_stay_in_their_places(zb, M, N, K, dtype):
    c = Linear(zb, M, N, K, dtype=dtype).run()
    sync(zb)
    plain = c.out.clone()
    c.X[2, 3], c.R[5, 7], c.bias[11] = INF, NAN, -INF
    c.W[:, 20] = NAN
    c.run()
    sync(zb)
    hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    hit[2, :], hit[5, 7], hit[:, 11], hit[:, 20] = True, True, True, True
    assert torch.equal(bits(c.out)[~hit], bits(plain)[~hit])
    assert not torch.isfinite(c.out[hit]).any()


@pytest.mark.parametrize("M,N,K", [(9, 72, 136), (2100, 2048, 128)])
@pytest.mark.parametrize("tanh", [False, True])
def test_linear_gelu_of_infinities(zb, M, N, K, tanh):
    """GeLU and GeLU' take their limits there, and nothing beside them changes."""
    c = Linear(zb, M, N, K, "gelu", tanh=tanh).run()
    sync(zb)
    plain = c.out.clone()
    c.bias[4], c.bias[5], c.bias[6] = INF, -INF, NAN
    c.run()
    sync(zb)
    rest = [n for n in range(N) if n not in (4, 5, 6)]
    assert torch.equal(bits(c.out)[:, rest], bits(plain)[:, rest])
    assert (c.out[:, 4] == INF).all() and torch.equal(c.out[:, 5], c.R[:, 5]) and torch.isnan(c.out[:, 6]).all()
    c = Linear(zb, M, N, K, "grad", tanh=tanh, transposed=True, residual=False).run()
    sync(zb)
    plain = c.out.clone()
    c.H[3, 4], c.H[3, 5], c.H[3, 6] = INF, -INF, NAN
    c.run()
    sync(zb)
    d = f64(c.X[3]) @ f64(c.W[4])
    near(c.out[3, 4], d, (K + 2) * 2.0 ** -23 * (np.abs(f64(c.X[3])) @ np.abs(f64(c.W[4]))) + 2.0 ** -8 * abs(d))
    assert c.out[3, 5] == 0 and torch.isnan(c.out[3, 6])
    same = bits(c.out) == bits(plain)
    same[3, 4:7] = True
    assert same.all()


@pytest.mark.parametrize("M,N,K,form,dtype", [(16, 1024, 4096, "store", BF16), (512, 1024, 1024, "grad", BF16),
                                              (2047, 2056, 520, "gelu", BF16), (300, 2048, 4096, "store", F32),
                                              (4096, 2048, 1024, "store", F32)])
def test_linear_captured_on_another_stream(zb, M, N, K, form, dtype):
    """Captured once, replayed on new inputs; the bits are the eager call's."""
    c = Linear(zb, M, N, K, form, dtype=dtype).run()
    sync(zb)
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        c.run()
    c.X.copy_(torch.randn(c.X.shape, device="cuda"))
    c.out.fill_(NAN)
    graph.replay()
    c.check()
    first = c.out.clone()
    c.out.fill_(NAN)
    st.wait_stream(torch.cuda.current_stream())
    c.run(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    sync(zb)
    assert torch.equal(bits(first), bits(c.out))


# --------------------------------------------------------------------- norm
def _norm_inputs(rows, width, dtype, seed=0, shift=0.5):
    rng = np.random.default_rng(seed + rows * 31 + width)
    X = dev(rng.normal(size=(rows, width)) * np.exp(0.5 * rng.normal(size=width)) + shift * rng.normal(size=width), dtype)
    gamma, beta = dev(1 + 0.2 * rng.normal(size=width)), dev(0.2 * rng.normal(size=width))
    return rng, X, gamma, beta


NORMS = [(1, 8), (2, 16), (5, 64), (3, 256), (33, 264), (7, 512), (100, 520), (16, 1024), (65, 1032), (9, 2048),
         (130, 2056), (257, 4096), (31, 5000), (8, 8192), (3, 12296), (2, 16384), (5, 16392), (2, 32768), (1025, 768),
         (40, 1400), (5, 10000), (700, 8), (1030, 4104)]
CHAIN = 64 + 5 + 16


def _near_forward(X, gamma, beta, eps, Y, mean, rstd):
    x, g, b = f64(X), f64(gamma), np.zeros(X.shape[1]) if beta is None else f64(beta)
    ref, m, r = oa.norm_forward(x, g, b, eps)
    dm = (CHAIN + 2) * E * np.abs(x).mean(axis=1)          # of the mean
    var = 1.0 / r ** 2                                       # with eps
    dr = (CHAIN + 8) * E + 1.01 * dm * dm / var              # of rstd, relative
    if mean is not None:
        near(mean, m, dm)
        near(rstd, r, r * dr)
    d = np.abs(x - m[:, None])
    off = np.abs(g) * r[:, None] * (dm[:, None] + (d + dm[:, None]) * (dr[:, None] + 4 * E)) + 4 * E * (np.abs(ref) + np.abs(b))
    near(Y, ref, off + 2.0 ** -8 * (np.abs(ref) + off))


@pytest.mark.parametrize("rows,width", NORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_forward(zb, rows, width, dtype):
    _, X, gamma, beta = _norm_inputs(rows, width, dtype)
    n = zb.make_layernorm(rows, width, zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32, eps=1e-5)
    Y, mean, rstd = empty_bf16(rows, width), empty_f32(rows), empty_f32(rows)
    zb.zb_layernorm_forward(n, X, gamma, beta, Y, mean, rstd)
    sync(zb)
    _near_forward(X, gamma, beta, n.eps, Y, mean, rstd)
    Y2 = empty_bf16(rows, width)
    zb.zb_layernorm_forward(n, X, gamma, None, Y2, None, None)
    sync(zb)
    _near_forward(X, gamma, None, n.eps, Y2, None, None)


def test_norm_forward_edges(zb):
    """Rows of one value, far from zero, tiny, of one infinity, of a NaN; each row by itself."""
    w = 264
    rng = np.random.default_rng(5)
    x = rng.normal(size=(8, w))
    x[0] = 3.0
    x[1] += 4096.0
    x[2] *= 1e-12
    x[3, 100] = INF
    x[4, 7] = NAN
    x[5] = 0.0
    x[6] *= 1e15
    X = dev(x, F32)
    gamma, beta = dev(np.ones(w)), dev(np.full(w, 0.25))
    n = zb.make_layernorm(8, w, zb.ZB_DT_F32, eps=1e-5)
    Y, mean, rstd = empty_bf16(8, w), empty_f32(8), empty_f32(8)
    zb.zb_layernorm_forward(n, X, gamma, beta, Y, mean, rstd)
    sync(zb)
    rows = [0, 1, 2, 5, 6, 7]
    _near_forward(X[rows], gamma, beta, n.eps, Y[rows], mean[rows], rstd[rows])
    assert torch.isnan(Y[4]).all() and torch.isnan(Y[3]).all()
    assert (Y[0] == 0.25).all() and (Y[5] == 0.25).all()


@pytest.mark.parametrize("rows,width", NORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_backward(zb, rows, width, dtype):
    rng, X, gamma, _ = _norm_inputs(rows, width, dtype, seed=1)
    dY, dR = dev(rng.normal(size=(rows, width))), dev(rng.normal(size=(rows, width)), dtype)
    n = zb.make_layernorm(rows, width, zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32)
    m, r = oa.norm_stats(f64(X), n.eps)
    mean, rstd = dev(m, F32), dev(r, F32)
    x, g, dy, m, r = f64(X), f64(gamma), f64(dY), f64(mean), f64(rstd)
    xh = np.abs((x - m[:, None]) * r[:, None])
    u = np.abs(dy * g)
    mu, along = u.mean(axis=1, keepdims=True), (u * xh).mean(axis=1, keepdims=True)

    def near_dx(got, ref, res, dtype):
        off = r[:, None] * E * (6 * (u + mu + xh * along) + CHAIN * mu + (CHAIN + 4) * xh * along)
        off = off + 2 * E * (np.abs(ref) + np.abs(res))
        near(got, ref, off + step(dtype) * (np.abs(ref) + off))

    dX, dX16 = torch.full_like(X, NAN), empty_bf16(rows, width)
    zb.zb_layernorm_backward_input(n, dY, X, gamma, mean, rstd, dR, dX, dX16)
    plain = torch.full_like(X, NAN)
    zb.zb_layernorm_backward_input(n, dY, X, gamma, mean, rstd, None, plain, None)
    there = dR.clone()
    zb.zb_layernorm_backward_input(n, dY, X, gamma, mean, rstd, there, there, None)  # in place
    sync(zb)
    ref = oa.norm_backward_input(dy, x, g, m, r, f64(dR))
    near_dx(dX, ref, f64(dR), dtype)
    near_dx(dX16, ref, f64(dR), BF16)
    near_dx(plain, oa.norm_backward_input(dy, x, g, m, r), np.zeros((1, width)), dtype)
    assert torch.equal(bits(there), bits(dX))
    if dtype == F32:
        assert torch.equal(bits(dX16), bits(dX.to(BF16)))

    dg, db = oa.norm_backward_weight(dy, x, m, r)
    chain = rows // 256 + 1 + 16
    off_g, off_b = (chain + 4) * E * (np.abs(dy) * xh).sum(axis=0), chain * E * np.abs(dy).sum(axis=0)
    dgamma, dbeta = empty_f32(width), empty_f32(width)
    zb.zb_layernorm_backward_weight(n, dY, X, mean, rstd, dgamma, dbeta, 0)
    only = empty_f32(width)
    zb.zb_layernorm_backward_weight(n, dY, X, mean, rstd, only, None, 0)
    sync(zb)
    near(dgamma, dg, off_g)
    near(dbeta, db, off_b)
    assert torch.equal(bits(only), bits(dgamma))
    old = dev(rng.normal(size=(2, width)), F32)
    sums = old.clone()
    zb.zb_layernorm_backward_weight(n, dY, X, mean, rstd, sums[0], sums[1], 1)
    sync(zb)
    assert torch.equal(sums[0], old[0] + dgamma) and torch.equal(sums[1], old[1] + dbeta)


def test_norm_no_rows(zb):
    n = zb.make_layernorm(0, 24)
    dg, db = dev(np.ones(24), F32), dev(np.ones(24), F32)
    zb.zb_layernorm_backward_weight(n, None, None, None, None, dg, db, 1)
    sync(zb)
    assert (dg == 1).all() and (db == 1).all()
    zb.zb_layernorm_backward_weight(n, None, None, None, None, dg, db, 0)
    sync(zb)
    assert (dg == 0).all() and (db == 0).all()


# ---------------------------------------------------------------- embedding
def _ids(tokens, vocab, kind, seed=0):
    rng = np.random.default_rng(seed + tokens + vocab)
    if kind == "same":
        return np.full(tokens, vocab - 1)
    if kind == "outside":
        return rng.choice([-1, -2 ** 31, vocab, 2 ** 31 - 1], size=tokens)
    if kind == "distinct":
        return rng.permutation(max(tokens, vocab))[:tokens] % vocab
    ids = np.minimum((np.exp(rng.random(tokens) * np.log(vocab + 1)) - 1).astype(np.int64), vocab - 1)
    ids = (ids * 7919) % vocab
    if kind == "padded":
        ids[rng.random(tokens) < 0.3] = rng.choice([-1, vocab])
    return ids


TOKENS = [1, 2, 31, 32, 33, 64, 65, 257, 1000, 1023, 1024, 1025, 1056, 4097, 8191, 20011]


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("vocab,kind", [(1, "falling"), (2, "padded"), (1000, "falling"), (1023, "same"),
                                        (1024, "padded"), (50021, "falling"), (3000, "distinct"), (64, "outside")])
def test_embedding(zb, tokens, vocab, kind):
    w = 8 * (1 + tokens % 5)
    k = TOKENS.index(tokens)
    dtype = (BF16, F32)[k % 2]
    ids = _ids(tokens, vocab, kind)
    rng = np.random.default_rng(tokens)
    e = zb.make_embedding(tokens, vocab, w, zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32, scale=1.7)
    table = dev(rng.normal(size=(vocab, w)))
    ids_d = i32(ids)
    Y = torch.full((tokens, w), NAN, dtype=dtype, device="cuda")
    zb.zb_embedding_forward(e, ids_d, table, Y)
    order, sid = i32(np.full(tokens, 77)), i32(np.full(tokens, 77))
    n = zb.zb_embedding_workspace_bytes(e)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    zb.zb_embedding_sort(e, ids_d, order, sid, ws, n)
    sync(zb)
    ref = oa.embedding(ids, f64(table), e.scale)
    near(Y, ref, (E + step(dtype)) * np.abs(ref))
    o, s = oa.embedding_order(ids, vocab)
    assert np.array_equal(order.cpu().numpy(), o) and np.array_equal(sid.cpu().numpy(), s)
    dY = dev(rng.normal(size=(tokens, w)), dtype)
    dE = empty_f32(vocab, w)
    zb.zb_embedding_backward(e, order, sid, dY, dE, 0, ws, n)
    again = empty_f32(vocab, w)
    zb.zb_embedding_backward(e, order, sid, dY, again, 0, ws, n)
    old = dev(rng.normal(size=(vocab, w)), F32)
    count = np.bincount(np.where((ids >= 0) & (ids < vocab), ids, vocab), minlength=vocab + 1)[:vocab]
    old[torch.from_numpy(count == 0).cuda()] = NAN  # rows that must not be touched
    more = old.clone()
    zb.zb_embedding_backward(e, order, sid, dY, more, 1, ws, n)
    sync(zb)
    ref = oa.embedding_backward(ids, vocab, f64(dY), e.scale)
    terms = oa.embedding_backward(ids, vocab, np.abs(f64(dY)), e.scale)
    off = (32 + count // 32 + 4)[:, None] * E * terms
    near(dE, ref, off)
    assert torch.equal(bits(dE), bits(again))
    near(more, f64(old) + ref, off + E * (np.abs(f64(old)) + np.abs(ref)) + E * terms)
    assert (ws[n:] == 255).all()


@pytest.mark.parametrize("tokens,vocab,w,dtype", [(700, 300, 1032, BF16), (700, 300, 2048, F32), (50, 20, 4104, BF16),
                                                  (100, 1 << 20, 8, F32), (3000, (1 << 21) + 5, 8, BF16)])
def test_embedding_wide(zb, tokens, vocab, w, dtype):
    ids = _ids(tokens, vocab, "padded", seed=3)
    rng = np.random.default_rng(4)
    e = zb.make_embedding(tokens, vocab, w, zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32, scale=-0.5)
    table = torch.randn((vocab, w), device="cuda").to(BF16)
    Y = torch.full((tokens, w), NAN, dtype=dtype, device="cuda")
    zb.zb_embedding_forward(e, i32(ids), table, Y)
    order, sid = i32(np.zeros(tokens)), i32(np.zeros(tokens))
    n = zb.zb_embedding_workspace_bytes(e)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    zb.zb_embedding_sort(e, i32(ids), order, sid, ws, n)
    dY = dev(rng.normal(size=(tokens, w)), dtype)
    dE = empty_f32(vocab, w)
    zb.zb_embedding_backward(e, order, sid, dY, dE, 0, ws, n)
    sync(zb)
    on = (ids >= 0) & (ids < vocab)
    at = np.unique(ids[on])
    ref = np.zeros((tokens, w))
    ref[on] = -0.5 * f64(table[torch.from_numpy(ids[on]).cuda()])
    near(Y, ref, 0.0 if dtype == F32 else 2.0 ** -8 * np.abs(ref))
    o, s = oa.embedding_order(ids, vocab)
    assert np.array_equal(order.cpu().numpy(), o) and np.array_equal(sid.cpu().numpy(), s)
    # the rows that occur, numbered by their places in `at`
    local = np.where(on, np.searchsorted(at, np.where(on, ids, at[0])), -1)
    got = dE[torch.from_numpy(at).cuda()]
    ref = oa.embedding_backward(local, len(at), f64(dY), -0.5)
    count = np.bincount(local[on], minlength=len(at))
    near(got, ref, (32 + count // 32 + 4)[:, None] * E * oa.embedding_backward(local, len(at), np.abs(f64(dY)), 0.5))
    rest = torch.ones(vocab, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(at).cuda()] = False
    assert not dE[rest].any()


def test_embedding_nan_stays_in_its_row(zb):
    ids = np.array([3, 1, 3, 3, 0, -1] * 40)
    e = zb.make_embedding(240, 5, 16, scale=2.0)
    dY = dev(np.ones((240, 16)))
    dY[5], dY[2, 3] = NAN, INF  # a padding token; a token of id 3
    order, sid = i32(np.zeros(240)), i32(np.zeros(240))
    n = zb.zb_embedding_workspace_bytes(e)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    zb.zb_embedding_sort(e, i32(ids), order, sid, ws, n)
    dE = empty_f32(5, 16)
    zb.zb_embedding_backward(e, order, sid, dY, dE, 0, ws, n)
    sync(zb)
    want = torch.tensor([80.0, 80.0, 0.0, 240.0, 0.0], device="cuda")[:, None].repeat(1, 16)
    want[3, 3] = INF
    assert torch.equal(dE, want)


def test_embedding_no_tokens(zb):
    e = zb.make_embedding(0, 70, 24)
    dE = empty_f32(70, 24)
    zb.zb_embedding_backward(e, None, None, None, dE, 0, None, 0)
    sync(zb)
    assert (dE == 0).all()


def test_embedding_foreign_order_stays_inside(zb):
    """Indices no sort has made: any sums, but nothing outside the buffers is touched."""
    T, V, w = 300, 40, 64
    e = zb.make_embedding(T, V, w)
    rng = np.random.default_rng(6)
    order = i32(rng.integers(-2 ** 31, 2 ** 31, T))
    sid = i32(rng.integers(-5, V + 5, T))
    n = zb.zb_embedding_workspace_bytes(e)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    big = torch.full((V + 2, w), 77.0, device="cuda")
    dY = dev(rng.normal(size=(T, w)))
    for accumulate in (0, 1):
        zb.zb_embedding_backward(e, order, sid, dY, big[1:-1], accumulate, ws, n)
        sync(zb)
    assert (big[0] == 77.0).all() and (big[-1] == 77.0).all() and (ws[n:] == 0).all()


def test_embedding_two_calls_at_once(zb):
    """Two streams with a workspace each, captured into graphs and replayed together."""
    T, V, w = 5000, 3000, 256
    e = zb.make_embedding(T, V, w)
    n = zb.zb_embedding_workspace_bytes(e)
    sets = []
    for k in range(2):
        s = dict(ids=i32(_ids(T, V, "padded", seed=k)), order=i32(np.zeros(T)), sid=i32(np.zeros(T)),
                 dY=dev(np.random.default_rng(k).normal(size=(T, w))), dE=empty_f32(V, w),
                 ws=torch.empty(n, dtype=torch.uint8, device="cuda"), graph=torch.cuda.CUDAGraph(),
                 stream=torch.cuda.Stream())

        def call(s=s):
            zb.zb_embedding_sort(e, s["ids"], s["order"], s["sid"], s["ws"], n)
            zb.zb_embedding_backward(e, s["order"], s["sid"], s["dY"], s["dE"], 0, s["ws"], n)

        call()
        sync(zb)
        s["alone"] = s["dE"].clone()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            call()
        sets.append(s)
    for s in sets:
        s["dE"].fill_(NAN)
    torch.cuda.synchronize()
    for _ in range(3):
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
    sync(zb)
    for s in sets:
        assert torch.equal(bits(s["dE"]), bits(s["alone"]))


# ------------------------------------------------------------ all together
@pytest.mark.parametrize("T,V,h,f,dtype,tanh", [(40, 100, 64, 256, F32, False), (1000, 700, 256, 1024, BF16, True),
                                                (2100, 5000, 512, 2048, F32, False)])
def test_first_stage(zb, T, V, h, f, dtype, tanh):
    """Embedding, then a pre-norm residual block: F, B and W as a pipeline's first
    stage runs them, every result against the oracle on the tensors that were read."""
    rng = np.random.default_rng(T)
    zdt = zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32
    act = zb.ZB_ACT_GELU_TANH if tanh else zb.ZB_ACT_GELU_ERF
    ids = _ids(T, V, "padded", seed=9)
    table, gamma, beta = dev(rng.normal(size=(V, h))), dev(1 + 0.1 * rng.normal(size=h)), dev(0.1 * rng.normal(size=h))
    W1, b1 = dev(rng.normal(size=(h, f)) / np.sqrt(h)), dev(0.1 * rng.normal(size=f))
    W2, b2 = dev(rng.normal(size=(f, h)) / np.sqrt(f)), dev(0.1 * rng.normal(size=h))
    dY, dY16 = dev(rng.normal(size=(T, h)), dtype), None
    dY16 = dY.to(BF16)
    R, Y = (torch.full((T, h), NAN, dtype=dtype, device="cuda") for _ in range(2))
    N, H, A, dH, dN = empty_bf16(T, h), empty_bf16(T, f), empty_bf16(T, f), empty_bf16(T, f), empty_bf16(T, h)
    mean, rstd = empty_f32(T), empty_f32(T)
    dR, dR16 = torch.full_like(R, NAN), empty_bf16(T, h)
    dW1, dW2, db1, db2 = empty_f32(h, f), empty_f32(f, h), empty_f32(f), empty_f32(h)
    dgamma, dbeta, dE = empty_f32(h), empty_f32(h), empty_f32(V, h)
    order, sid = i32(np.zeros(T)), i32(np.zeros(T))
    e = zb.make_embedding(T, V, h, zdt, scale=float(np.sqrt(h)))
    n = zb.make_layernorm(T, h, zdt)
    ws = torch.empty(zb.zb_embedding_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    # F
    zb.zb_embedding_forward(e, i32(ids), table, R)
    zb.zb_layernorm_forward(n, R, gamma, beta, N, mean, rstd)
    zb.zb_linear_product(zb.make_linear(T, f, h, epilogue=zb.ZB_LINEAR_GELU, act=act), N, W1, b1, None, None, H, A)
    zb.zb_linear_product(zb.make_linear(T, h, f, dtype=zdt), A, W2, b2, R, None, Y, None)
    # B
    zb.zb_linear_product(zb.make_linear(T, f, h, transposed=True, epilogue=zb.ZB_LINEAR_GELU_GRAD, act=act), dY16, W2,
                         None, None, H, dH, None)
    zb.zb_linear_product(zb.make_linear(T, h, f, transposed=True), dH, W1, None, None, None, dN, None)
    zb.zb_layernorm_backward_input(n, dN, R, gamma, mean, rstd, dY, dR, dR16)
    # W
    zb.zb_backward_weight(zb.make_block(T, f, h, act=zb.ZB_ACT_NONE, has_bias=True), A, None, None, dY16, dW2, None, db2,
                          None, 0)
    zb.zb_backward_weight(zb.make_block(T, h, f, act=zb.ZB_ACT_NONE, has_bias=True), N, None, None, dH, dW1, None, db1,
                          None, 0)
    zb.zb_layernorm_backward_weight(n, dN, R, mean, rstd, dgamma, dbeta, 0)
    zb.zb_embedding_sort(e, i32(ids), order, sid, ws, ws.numel())
    zb.zb_embedding_backward(e, order, sid, dR, dE, 0, ws, ws.numel())
    sync(zb)

    def close(got, ref, tol):
        assert np.linalg.norm(f64(got) - ref) <= tol * np.linalg.norm(ref)

    half = 2.0 ** -8  # every value off by half a bf16 step at most
    close(R, oa.embedding(ids, f64(table), e.scale), half)
    close(N, oa.norm_forward(f64(R), f64(gamma), f64(beta), n.eps)[0], half)
    a, d = oa.linear(f64(N), f64(W1), form="gelu", bias=f64(b1), tanh=tanh)
    close(H, d, half)
    close(A, a, half)
    close(Y, oa.linear(f64(A), f64(W2), bias=f64(b2), R=f64(R))[0], half)
    close(dH, oa.linear(f64(dY16), f64(W2), True, "grad", H=f64(H), tanh=tanh)[0], half)
    close(dN, oa.linear(f64(dH), f64(W1), True)[0], half)
    close(dR, oa.norm_backward_input(f64(dN), f64(R), f64(gamma), f64(mean), f64(rstd), f64(dY)), half)
    dg, db = oa.norm_backward_weight(f64(dN), f64(R), f64(mean), f64(rstd))
    close(dgamma, dg, 1e-5)
    close(dbeta, db, 1e-5)
    close(dW2, f64(A).T @ f64(dY16), 1e-5)
    close(dW1, f64(N).T @ f64(dH), 1e-5)
    close(dE, oa.embedding_backward(ids, V, f64(dR), e.scale), 1e-6)
    # and the whole chain from its inputs: every stored tensor is rounded once, so
    # the ends are within a few roundings of the exact chain
    R0 = oa.embedding(ids, f64(table), e.scale)
    N0, m0, r0 = oa.norm_forward(R0, f64(gamma), f64(beta), n.eps)
    A0, H0 = oa.linear(N0, f64(W1), form="gelu", bias=f64(b1), tanh=tanh)
    Y0 = oa.linear(A0, f64(W2), bias=f64(b2), R=R0)[0]
    dH0 = oa.linear(f64(dY16), f64(W2), True, "grad", H=H0, tanh=tanh)[0]
    dN0 = oa.linear(dH0, f64(W1), True)[0]
    dR0 = oa.norm_backward_input(dN0, R0, f64(gamma), m0, r0, f64(dY))
    close(Y, Y0, 4 * half)
    close(dR, dR0, 6 * half)
    close(dE, oa.embedding_backward(ids, V, dR0, e.scale), 6 * half)
