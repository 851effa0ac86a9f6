"""The calls for several continuations of one prompt in the bounds-checking build: every checked
index inside its buffer."""
import pytest
import test_gpu_beam as beam
import test_gpu_prefix_attn as attn
import test_gpu_rope as rope
from gpu_util import torch_cuda

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


@pytest.mark.parametrize("case", range(len(attn.CASES)))
def test_attention_stays_in_bounds(torch, case):
    sizes, shared, own, Hq, Hkv, D, page = attn.CASES[case]
    attn.check(torch, attn.problem(torch, sizes, shared, own, Hq, Hkv, D, page, torch.bfloat16))
    assert q4.q4gemv_bounds_violations() == 0


def test_attention_with_limits_stays_in_bounds(torch):
    attn.test_limits_of_any_kind(torch)
    attn.test_contents_that_make_no_sense_stay_in_bounds(torch)
    attn.test_causal_prompt(torch, 300, 1, 2, 2, 64, 128)
    assert q4.q4gemv_bounds_violations() == 0


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,half", [(33, 14, 2, 64, 32, False), (5, 6, 2, 96, 48, True), (2, 3, 1, 17, 16, False),
                                                 (3, 2, 1, 256, 256, True), (1500, 32, 8, 128, 128, True)])
def test_rope_stays_in_bounds(torch, T, Hq, Hkv, D, rot, half):
    for dtype in (torch.float32, torch.bfloat16):
        rope.check(torch, T, Hq, Hkv, D, rot, half, dtype, torch.float16, drop=0.2, layout="paired", odd=1)
        rope.check(torch, T, Hq, Hkv, D, rot, half, dtype, torch.bfloat16, drop=0.2, layout="tokens")
    assert q4.q4gemv_bounds_violations() == 0


@pytest.mark.parametrize("groups,W,K,V", [(1, 1, 1, 1), (3, 2, 5, 31), (2, 4, 8, 4097), (2, 32, 32, 40001), (300, 2, 2, 130)])
def test_beam_step_stays_in_bounds(torch, groups, W, K, V):
    beam.test_beam_step_against_the_definition(torch, groups, W, K, V)
    beam.test_rows_of_any_stride_and_alignment(torch)
    assert q4.q4gemv_bounds_violations() == 0


def test_reorder_stays_in_bounds(torch):
    beam.test_reorder_against_the_definition(torch, "tokens", 3, 3, 5, 3, 7, 9, 3, "float16")
    beam.test_reorder_against_the_definition(torch, "heads", 1, 4, 48, 2, 16, 64, 16, "bfloat16")
    beam.test_reorder_leaves_pages_outside_the_pool_alone(torch)
    assert q4.q4gemv_bounds_violations() == 0
