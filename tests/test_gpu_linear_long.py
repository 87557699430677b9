"""fp32 products of a long K: what each accumulator holds, and in what order the
sums are added.

The operands stay on the GPU (some are hundreds of MB); the values they are compared
with are computed there in 64 bits by plain products.  Element-wise bounds as in
test_gpu_around.py: K products are off by at most K 2^-23 times the sum of the
absolute products, and the norm of the error is a random walk, below 1e-6 of the
norm of the result, whatever K, since an accumulator takes 512 products.
"""

import pytest
import torch

from tests.gpu_util import have_gpu, sync

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
NAN = float("nan")


@pytest.fixture(scope="module")
def zb():
    if not have_gpu():
        pytest.skip("no CUDA device")
    from split_backward_gemms_gb300 import build as B
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


def normal(shape, seed, std=1.0, dtype=BF16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda", dtype=F32) * std).to(dtype)


def product(X, W):
    """X W and |X| |W| in 64 bits, by columns of W so that its copy stays small."""
    D = torch.empty((X.shape[0], W.shape[1]), dtype=F64, device="cuda")
    A = torch.empty_like(D)
    x = X.to(F64)
    for c in range(0, W.shape[1], 2048):
        w = W[:, c:c + 2048].to(F64)
        D[:, c:c + 2048], A[:, c:c + 2048] = x @ w, x.abs() @ w.abs()
    return D, A


def fp32_product(zb, X, W, transposed=False, bias=None, R=None):
    N = W.shape[0] if transposed else W.shape[1]
    out = torch.full((X.shape[0], N), NAN, dtype=F32, device="cuda")
    zb.zb_linear_product(zb.make_linear(X.shape[0], N, X.shape[1], transposed=transposed, dtype=zb.ZB_DT_F32), X, W, bias,
                         R, None, out, None)
    return out


def check_random(zb, M, N, K, transposed):
    X, W = normal((M, K), M + K), normal((K, N), N, K ** -0.5)
    out = fp32_product(zb, X, W.T.contiguous() if transposed else W, transposed)
    sync(zb)
    D, A = product(X, W)
    off = (out.to(F64) - D).abs()
    assert (off <= (K + 2) * 2.0 ** -23 * A).all()
    assert torch.linalg.norm(off) <= 1e-6 * torch.linalg.norm(D)


# blocks of 64 along K a CTA takes that 16 accumulators of equal length do not divide
# evenly: 129, 145, 161 (one part of K), 129 (8 parts)
@pytest.mark.parametrize("M,N,K", [(16, 16384, 8256), (5, 20488, 9280), (32, 16384, 10304), (16, 256, 66048)])
@pytest.mark.parametrize("transposed", [False, True])
def test_nothing_is_added_that_no_product_wrote(zb, M, N, K, transposed):
    """Large sums left in every SM's tensor memory by the call before do not show."""
    big = torch.full((32, 8192), 100.0, dtype=BF16, device="cuda")
    wide = torch.full((8192, 19456), 100.0, dtype=BF16, device="cuda")  # a tile of 128 columns for each of 152 SMs
    left = fp32_product(zb, big, wide)
    check_random(zb, M, N, K, transposed)
    assert (left == 8192 * 1e4).all()


# few rows and few tiles, whose kernel splits K among CTAs or not at all
LONG = [(16, 16384, 16384), (32, 19456, 8704), (64, 16384, 8192), (64, 16384, 16384), (128, 8192, 8192), (512, 2048, 8192),
        (512, 2048, 16384), (16, 1024, 65536)]


@pytest.mark.parametrize("M,N,K", LONG)
@pytest.mark.parametrize("transposed", [False, True])
def test_long_k(zb, M, N, K, transposed):
    check_random(zb, M, N, K, transposed)


@pytest.mark.parametrize("M,N,K", LONG + [(2048, 4096, 8192)])
@pytest.mark.parametrize("transposed", [False, True])
def test_an_accumulator_takes_512_products(zb, M, N, K, transposed):
    """2^31, K - 2 halves, -2^31: beside 2^31 an accumulator loses halves (at most the 511
    that it takes; where its magnitude is cut to a step of 128 just below 2^31, it may
    gain up to 127), but every other one is exact, and so are the fp32 sums of what is
    left, multiples of 128 below 2^31 and of 256 above.  (Every CTA's part of K is a
    multiple of 512 here.)"""
    X, W = torch.ones((M, K), dtype=BF16, device="cuda"), torch.full((K, N), 0.5, dtype=BF16, device="cuda")
    X[:, 0], X[:, -1] = 2.0 ** 16, 2.0 ** 16
    W[0], W[-1] = 2.0 ** 15, -2.0 ** 15
    out = fp32_product(zb, X, W.T.contiguous() if transposed else W, transposed)
    sync(zb)
    lost = (K - 2) / 2 - out
    assert lost.min() >= -127 and lost.max() <= 511
    assert (out == out[0, 0]).all()


# the kernel for few rows or tiles (the first two), and the other one
@pytest.mark.parametrize("M,N,K", [(48, 512, 8192), (300, 512, 8192), (2048, 2048, 8192), (2051, 2056, 8200), (2048, 2048, 512),
                                   (2048, 2048, 1000)])
@pytest.mark.parametrize("transposed", [False, True])
def test_a_large_residual_is_rounded_three_times_at_most(zb, M, N, K, transposed):
    """Sums of 512 products are 0.3 of a step of the residual, so each would be lost by
    itself; together they are not.  Three roundings at the size of the result, whatever K."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + K)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    X = uniform(0.5, 1.5, M, K).to(BF16)
    W = (uniform(0.5, 1.5, K, N) * (0.3 * 2.0 ** -3 / 512)).to(BF16)
    R, bias = uniform(2.0 ** 20, 2.0 ** 21, M, N), uniform(-0.05, 0.05, N).to(BF16)
    out = fp32_product(zb, X, W.T.contiguous() if transposed else W, transposed, bias, R)
    sync(zb)
    D, A = product(X, W)
    ref = D + bias.to(F64) + R.to(F64)
    assert ((out.to(F64) - ref).abs() <= 3 * 2.0 ** -24 * ref.abs() + (K + 2) * 2.0 ** -23 * A).all()
