"""Host-side checks of the mixture-of-experts calls beyond test_moe_api.py.  Every call below
fails a check that runs before the first CUDA call, or is an empty problem."""
import pytest
from test_moe_api import INV, OK, UNS, block, gemm, route

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build


@pytest.fixture(scope="module")
def L():
    q4build.build()
    return q4.lib()


def test_bias_on_the_score_is_a_score_of_its_own(L):
    flag = q4.Q4_ROUTE_SCORE_BIAS
    for kind in (q4.Q4_ROUTE_SOFTMAX, q4.Q4_ROUTE_SIGMOID):
        assert route(L, T=0, score=kind | flag) == OK and block(L, T=0, score=kind | flag) == OK
    for bad in (flag | 2, flag << 1, -1, flag | 0x100):
        assert route(L, score=bad) == INV and block(L, score=bad) == INV


def test_products_refuse_long_rows_before_anything_is_launched(L):
    """K above 2^26: no workspace, and the block refuses before its router's launch (with the
    addresses below a launch would be an error of another kind)."""
    K = 1 << 27
    far = [(i + 1) << 44 for i in range(20)]   # disjoint however long the arrays are
    assert L.q4moe_gemm_workspace(8, 4, 64, K, 4, 0) == -1
    assert L.q4moe_gemm_workspace(8, 4, 64, 1 << 26, 4, 0) > 0
    assert gemm(L, K=K, ws=1 << 40, codes=far[0], scales=far[1], zeros=far[2], x=far[3], rows=far[4], offsets=far[5],
                y=far[6], work=far[7]) == UNS
    assert L.q4moe_gemm_workspace(8, 2 ** 31 - 1, 64, 64, 4, 0) == -1
    names = ("up_codes", "up_scales_f16", "up_zeros_u4_or_null", "down_codes", "down_scales_f16",
             "down_zeros_u4_or_null", "logits", "bias_or_null", "token_mask_or_null", "a", "x", "post_gamma", "gate",
             "pre_gamma", "ids", "route_weights", "out", "out_norm", "workspace")
    assert L.q4moe_block_workspace(1, 1, 1, 32, K, 0) == -1
    assert block(L, T=1, E=1, top_k=1, H=32, inner=K, workspace_bytes=1 << 40, **dict(zip(names, far))) == UNS
