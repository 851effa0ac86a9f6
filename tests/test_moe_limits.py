"""Host-side checks of the mixture-of-experts calls beyond test_moe_api.py.  Every call below
fails a check that runs before the first CUDA call, or is an empty problem."""
import pytest
from test_moe_api import INV, OK, block, route

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
