"""The example's block on the library as it is shipped.  (test_gpu_moe.py checks it after a
module-wide switch to the bounds-checking build.)"""
import os
import sys

import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype,limit", [("float32", 1e-5), ("bfloat16", 4 * 2.0 ** -8)])
def test_example_block_on_the_shipped_library(dtype, limit):
    torch = torch_cuda()
    import moe_block
    assert q4.lib()._name == q4build.LIB_PATH
    assert moe_block.check(getattr(torch, dtype), hidden=512, inner=256, experts=8, top_k=2, group=64) <= limit
