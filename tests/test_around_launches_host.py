"""What the operators around the block ask of the CUDA runtime (no GPU: a stand-in
takes the calls)."""

import ctypes as C

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


CALLS = f"""
from split_backward_gemms_gb300 import zb
n = zb.make_layernorm(64, 512)
zb.zb_layernorm_forward(n, {P}, {P}, {P}, {P}, {P}, {P}, stream=0)
zb.zb_layernorm_backward_input(n, {P}, {P}, {P}, {P}, {P}, {P}, {P}, None, stream=0)
zb.zb_layernorm_backward_weight(n, {P}, {P}, {P}, {P}, {P}, {P}, 0, stream=0)
for tokens in (100, 3000, 9000):
    e = zb.make_embedding(tokens, 1000, 64)
    zb.zb_embedding_forward(e, {P}, {P}, {P}, stream=0)
    zb.zb_embedding_sort(e, {P}, {P}, {P}, {P}, 1 << 40, stream=0)
    zb.zb_embedding_backward(e, {P}, {P}, {P}, {P}, 0, {P}, 1 << 40, stream=0)
for M in (16, 2000):
    zb.zb_linear_product(zb.make_linear(M, 2048, 512), {P}, {P}, {P}, {P}, None, {P}, None, stream=0)
zb.zb_moe_forward(zb.make_moe(64, 128, 256, 4), {P}, {P}, {P}, {P}, {P}, {P}, {P}, {P}, {P}, stream=0)
"""


@pytest.mark.parametrize("env,programmatic", [({}, 1), ({"ZB_GEMM_PDL": "1"}, 1), ({"ZB_GEMM_PDL": "0"}, 0)])
def test_programmatic_launches_as_the_environment_says(folder, env, programmatic):
    launches = cudart_shim.run(folder, CALLS, **env)
    # norm 3; lookup, order, gradient and join each three times; linear 2; experts' two products
    assert len(launches) == 3 + 12 + 2 + 2 and {n[3] for n in launches} == {programmatic}


class LinearArgs(C.Structure):
    """The last argument of the kernel for many rows (csrc/linear.cu)."""
    _fields_ = [("pointers", C.c_void_p * 5), ("ld", C.c_int64 * 3), ("MNK", C.c_int32 * 3), ("save", C.c_int32),
                ("tanh", C.c_int32), ("hint_a", C.c_int32), ("hint_b", C.c_int32), ("hint_out", C.c_int32),
                ("hint_once", C.c_int32), ("tile_n", C.c_int32)]


LINEAR = f"""
from split_backward_gemms_gb300 import zb
g = zb.make_linear(8192, 4096, 4096, transposed=True, epilogue=zb.ZB_LINEAR_GELU_GRAD)
zb.zb_linear_product(g, {P}, {P}, None, {P}, {P}, {P}, None, stream=0)
"""


@pytest.mark.parametrize("env,once", [({}, 1), ({"ZB_GEMM_L2_HINTS": "0"}, 0)])
def test_l2_priorities_of_linear_maps_as_the_environment_says(folder, env, once):
    (launch,) = cudart_shim.run(folder, LINEAR, SHIM_ARG="5", SHIM_BYTES=str(C.sizeof(LinearArgs)), **env)
    a = LinearArgs.from_buffer_copy(launch[4])
    assert list(a.MNK) == [8192, 4096, 4096] and a.tile_n == 256 and a.hint_once == once
    assert (a.hint_a, a.hint_b, a.hint_out) != (0, 0, 0) if once else (a.hint_a, a.hint_b, a.hint_out) == (0, 0, 0)
