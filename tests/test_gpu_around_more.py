"""More of the operators around the block against the fp64 oracle (bounds as in
test_gpu_around.py)."""

import numpy as np
import pytest
import torch

from oracle import around as oa
from tests import cudart_shim
from tests.gpu_util import f64, have_gpu, sync
from tests.test_gpu_around import Linear, _ids, i32

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
