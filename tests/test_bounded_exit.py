"""A kernel that gives up on a bounded wait must not leave its bulk copies in flight: they
would land in shared memory that the next CTA owns.  Any role may give up at any moment, so
the copying lane waits for its copies whether or not a flag is raised when it looks.

Read from the sources: the race needs a wait that expires while a copy is under way, which no
run shows reliably.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_decode_gb300", "csrc")
FLAG = r"if \((?:\*abort_flag|aborted\(\))\)"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["moe_gemm_few.cuh", "moe_gemm_many.cuh", "q4gemm.cu", "q4gemm_split.cu",
                                  "q4gemv_tc.cu", "q4gemv_stream_kernel.cuh"])
def test_copies_are_drained_whatever_the_flag(name):
    text = source(name)
    drains = list(re.finditer(r"mbar_wait\((?:code_full|full_a|cfull|full)\([^;]*50ull \* 1000 \* 1000\);", text))
    assert len(drains) == 1, "the copying warp waits for the copies it issued"
    before = text[:drains[0].start()]
    last_copy = max(before.rfind("tma_load_2d("), before.rfind("bulk_copy("))
    assert last_copy > 0 and not re.search(FLAG, before[last_copy:]), "the drain depends on a flag"


@pytest.mark.parametrize("name", ["q4gemm.cu", "q4gemm_split.cu", "q4gemv_tc.cu"])
def test_tensor_memory_is_freed_behind_the_last_product(name):
    """The same for the products still writing the tensor memory that a CTA frees as it ends."""
    text = source(name)
    teardown = text.rindex("mbar_wait(done_bar, 0")
    assert teardown < text.index("tcgen05.dealloc")
    condition = text[text.rindex("if (", 0, teardown):teardown]
    assert "warp == 1 && lane == 0" in condition and "abort_flag" not in condition
