"""The mixture-of-experts operators in the bounds-checking build, the products on the paths of
test_gpu_moe_paths.py: every checked index inside its buffer."""
import numpy as np
import pytest
from gpu_util import torch_cuda
from test_gpu_moe import check_norm, check_route, num, within
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


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (17, 33, 5), (129, 64, 8), (65, 1000, 32), (1031, 128, 8), (6000, 24, 32)])
def test_router_stays_in_bounds(torch, T, E, k):
    k = min(k, E)
    rng = np.random.default_rng(T)
    logits = rng.normal(0, 2, (T, E)).astype(np.float32)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    check_route(torch, logits, k, "sigmoid", True, bias=rng.normal(0, 1, E).astype(np.float32), mask=mask)
    assert q4.q4gemv_bounds_violations() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,H,k", [(1, 1, 1), (2, 7, 2), (5, 896, 0), (9, 1002, 3), (33, 2047, 4), (3, 16384, 1), (2, 16383, 2)])
def test_norm_stays_in_bounds(torch, bf16, T, H, k):
    check_norm(torch, T + H, T, H, k, bf16, True, "token", True)
    check_norm(torch, T + H, T, H, k, bf16, False, "channel", True, odd_gate=True)
    assert q4.q4gemv_bounds_violations() == 0
