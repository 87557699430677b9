"""More of the operators around the block against the fp64 oracle (bounds as in
test_gpu_around.py)."""

import numpy as np
import pytest
import torch

from oracle import around as oa
from tests import cudart_shim
from tests.gpu_util import empty_f32, f64, have_gpu, sync
from tests.test_gpu_around import BF16, E, F32, Linear, _ids, _norm_inputs, dev, i32, near

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


# 131072 tokens and more: a warp of the cluster of 16 (65536: of 8) has more of them than it holds in registers
SORTED = [(20011, 50021), (70001, 1 << 20), (131073, 1000), (262147, 32000), (300001, 2)]


def sort_all(zb):
    for tokens, vocab in SORTED:
        ids = _ids(tokens, vocab, "padded", seed=11)
        e = zb.make_embedding(tokens, vocab, 8)
        n = zb.zb_embedding_workspace_bytes(e)
        ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
        order, sid = i32(np.full(tokens, 77)), i32(np.full(tokens, 77))
        zb.zb_embedding_sort(e, i32(ids), order, sid, ws, n)
        sync(zb)
        o, s = oa.embedding_order(ids, vocab)
        assert np.array_equal(order.cpu().numpy(), o) and np.array_equal(sid.cpu().numpy(), s)
        assert (ws[n:] == 255).all()


def test_many_tokens_sorted(zb):
    sort_all(zb)


def test_many_tokens_sorted_without_clusters_of_16(zb, tmp_path):
    code = "from split_backward_gemms_gb300 import zb; import tests.test_gpu_around_more as t; t.sort_all(zb)"
    for most, blocks in ((16, 16), (8, 8)):
        launches = cudart_shim.run(tmp_path, code, fake=False, SHIM_CLUSTERS=str(most))
        assert [n[:2] for n in launches] == [(blocks, 1024)] * len(SORTED)


def _bits_child(out):
    """Chains of the library's kernels, each reading what the one before it wrote."""
    from split_backward_gemms_gb300 import zb
    got = {}
    for T, h, f, zdt, dt in ((40, 64, 256, zb.ZB_DT_F32, torch.float32), (2100, 512, 2048, zb.ZB_DT_BF16, torch.bfloat16)):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(T)

        def normal(*shape, dtype=torch.bfloat16):
            return torch.randn(shape, generator=gen, device="cuda").to(dtype)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        e, n = zb.make_embedding(T, 700, h, zdt, scale=2.0), zb.make_layernorm(T, h, zdt)
        ids, table, gamma, W1, W2 = i32(_ids(T, 700, "padded")), normal(700, h), normal(h), normal(h, f), normal(f, h)
        R, R2, N, H, A, dN = empty(T, h, dtype=dt), empty(T, h, dtype=dt), empty(T, h), empty(T, f), empty(T, f), empty(T, h)
        mean, rstd, dg, dE = (empty(*s, dtype=torch.float32) for s in ((T,), (T,), (h,), (700, h)))
        order, sid = empty(T, dtype=torch.int32), empty(T, dtype=torch.int32)
        dR, ws = empty(T, h, dtype=dt), empty(zb.zb_embedding_workspace_bytes(e), dtype=torch.uint8)
        torch.cuda.synchronize()
        zb.zb_embedding_forward(e, ids, table, R)
        zb.zb_layernorm_forward(n, R, gamma, None, N, mean, rstd)
        zb.zb_linear_product(zb.make_linear(T, f, h, epilogue=zb.ZB_LINEAR_GELU), N, W1, None, None, None, H, A)
        zb.zb_linear_product(zb.make_linear(T, h, f, dtype=zdt), A, W2, None, R, None, R2, None)
        zb.zb_linear_product(zb.make_linear(T, h, f, transposed=True), H, W1, None, None, None, dN, None)
        zb.zb_layernorm_backward_input(n, dN, R2, gamma, mean, rstd, R, dR, None)
        zb.zb_layernorm_backward_weight(n, dN, R2, mean, rstd, dg, None, 0)
        zb.zb_embedding_sort(e, ids, order, sid, ws, ws.numel())
        zb.zb_embedding_backward(e, order, sid, dR, dE, 0, ws, ws.numel())
        sync(zb)
        for name, t in dict(R2=R2, H=H, A=A, dR=dR, dg=dg, dE=dE, order=order).items():
            got[f"{name}_{T}"] = t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()
    np.savez(out, **got)


def test_launch_modes_change_no_bits(zb, tmp_path):
    """Programmatic launches, and the L2 priorities of the products' copies, on and off."""
    res = []
    for k, env in enumerate(({}, {"ZB_GEMM_PDL": "0"}, {"ZB_GEMM_L2_HINTS": "0"})):
        out = str(tmp_path / f"{k}.npz")
        launches = cudart_shim.run(tmp_path, f"import tests.test_gpu_around_more as t; t._bits_child({out!r})", fake=False,
                                   **env)
        assert {n[3] for n in launches} == {0 if "ZB_GEMM_PDL" in env else 1}
        res.append(np.load(out))
    for other in res[1:]:
        for name in res[0].files:
            assert np.array_equal(res[0][name], other[name]), (name, other)


# rows that a thread of the norm's W adds one after the other: 9 to 47
@pytest.mark.parametrize("rows,width", [(1000, 16392), (500, 32768), (3000, 8200), (2300, 12296), (4700, 4104), (9000, 264),
                                        (4097, 2056)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_weight_of_many_rows(zb, rows, width, dtype):
    """A column's roundings: one for each row a thread adds, then the shuffles, warps and
    blocks that hold the column; dgamma's terms have two of their own."""
    rng, X, _, _ = _norm_inputs(rows, width, dtype, seed=2)
    dY = dev(rng.normal(size=(rows, width)))
    n = zb.make_layernorm(rows, width, zb.ZB_DT_BF16 if dtype == BF16 else zb.ZB_DT_F32)
    m, r = oa.norm_stats(f64(X), n.eps)
    mean, rstd = dev(m, F32), dev(r, F32)
    old = dev(rng.normal(size=(2, width)), F32)
    sums, more = empty_f32(2, width), old.clone()
    zb.zb_layernorm_backward_weight(n, dY, X, mean, rstd, sums[0], sums[1], 0)
    zb.zb_layernorm_backward_weight(n, dY, X, mean, rstd, more[0], more[1], 1)
    sync(zb)
    x, dy, m, r = f64(X), f64(dY), f64(mean), f64(rstd)
    vecs = 4  # of 8 columns, that a cluster of 8 blocks of 512 threads takes
    while width > 256 * vecs:
        vecs *= 2
    chain = -(-rows * vecs // 4096) + max(0, 5 - int(np.log2(vecs))) + 16 // max(1, vecs // 32) + 8
    dg, db = oa.norm_backward_weight(dy, x, m, r)
    size = (np.abs(dy) * np.abs((x - m[:, None]) * r[:, None])).sum(axis=0)
    near(sums[0], dg, (chain + 2) * E * size)
    near(sums[1], db, chain * E * np.abs(dy).sum(axis=0))
    assert torch.equal(more, old + sums)
