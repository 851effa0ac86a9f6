"""Host-side limits of the calls for several continuations of one prompt: sizes whose products
would pass 64 bits are refused.  No pointer here is dereferenced."""
import pytest
import test_decode_api as api

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build


@pytest.fixture(scope="module")
def L():
    q4build.build()
    return q4.lib()


def test_page_tables_of_a_reordering(L):
    """4 n max_pages bytes are compared with the other arrays: 2^30 x 4 x (2^31 - 1) is 2^63."""
    most = 2 ** 31 - 1
    for groups, W, columns in ((2 ** 20, 1024, most), (2 ** 21 - 1, 1024, most), (16, 1024, 2 ** 30)):
        assert api.reorder(L, groups=groups, W=W, max_pages=columns) == api.UNS, (groups, W, columns)
    # what is accepted is looked at as a whole: tables that reach into the arrays behind them
    assert api.reorder(L, groups=2 ** 12, W=2, max_pages=2 ** 20) == api.INV
