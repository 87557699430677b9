"""What the operators around the block ask of the CUDA runtime (no GPU: a stand-in
takes the calls)."""

import pytest

from tests import cudart_shim

P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def folder(tmp_path_factory):
    return tmp_path_factory.mktemp("shim")


SORT = f"""
from split_backward_gemms_gb300 import zb
for tokens in (300, 8192, 8193, 200000):
    e = zb.make_embedding(tokens, 32000, 64)
    zb.zb_embedding_sort(e, {P}, {P}, {P}, {P}, 1 << 40, stream=0)
"""


@pytest.mark.parametrize("most,blocks", [(16, [8, 8, 16, 16]), (8, [8, 8, 8, 8])])
def test_sort_takes_clusters_that_can_be_resident(folder, most, blocks):
    assert [n[0] for n in cudart_shim.run(folder, SORT, SHIM_CLUSTERS=str(most))] == blocks
