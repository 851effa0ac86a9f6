"""The expert products in the bounds-checking build, on the paths of test_gpu_moe_paths.py:
every checked index inside its buffer."""
import pytest
from gpu_util import torch_cuda
from test_gpu_moe import num, within
from test_gpu_moe_paths import SHARED, shared_call

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_cuda()
    path = q4build.build(variant="check")
    saved = q4._lib, q4.library_path
    q4._lib, q4.library_path = None, lambda: path
    try:
        assert q4.q4gemv_bounds_violations() == 0   # a checking build, counter clear
        yield t
    finally:
        q4._lib, q4.library_path = saved


@pytest.mark.parametrize("counts,N,K,g,bf16,nt", SHARED)
def test_shared_items_stay_in_bounds(torch, counts, N, K, g, bf16, nt):
    call, want, bound, *_ = shared_call(torch, counts, N, K, g, False, False, bf16, True)
    within(num(call()), want, bound, "y")
    assert q4.q4gemv_bounds_violations() == 0


@pytest.mark.parametrize("K,g", [(1120, 32), (2112, 64)])
def test_several_chunks_of_scales_stay_in_bounds(torch, K, g):
    call, want, bound, *_ = shared_call(torch, [130, 2, 0, 71], 300, K, g, False, True, True, True)
    within(num(call()), want, bound, "y")
    assert q4.q4gemv_bounds_violations() == 0
