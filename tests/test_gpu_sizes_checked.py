"""The sizes that take other ways through the attention's plan and the beam step, in the
bounds-checking build: every checked index inside its buffer."""
import pytest
import test_gpu_attn_sizes as attn
import test_gpu_beam_sizes as beam
from test_gpu_decode_checked import torch  # noqa: F401  (the fixture: the checking build in the product's place)

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,most,Hq,Hkv", [attn.GROUPS[i] for i in (0, 2, 5, 6)])
def test_numbers_of_groups_stay_in_bounds(torch, groups, most, Hq, Hkv):  # noqa: F811
    for own, kind in ((False, "limits"), (True, "plain")):
        attn.test_numbers_of_groups(torch, groups, most, Hq, Hkv, own, kind)
    assert q4.q4gemv_bounds_violations() == 0


def test_runs_segments_and_parts_stay_in_bounds(torch):  # noqa: F811
    attn.test_numbers_of_runs(torch, [3] * 700, False, "limits")
    attn.test_numbers_of_runs(torch, [3, 0, 5, 1] * 250, True, "plain")
    attn.test_many_segments_a_cta(torch)
    attn.test_rows_of_many_parts(torch, 3, 14, 2, 64)
    attn.test_rows_of_many_parts(torch, 20, 14, 2, 64)
    assert q4.q4gemv_bounds_violations() == 0


def test_beam_sizes_stay_in_bounds(torch):  # noqa: F811
    beam.test_more_rows_than_65535(torch, 2100, 32, 4, 2)
    beam.test_chunks_of_several_parts(torch, 620, 10, 8, 70001)
    beam.test_logits_whose_scores_round_alike(torch)
    assert q4.q4gemv_bounds_violations() == 0
