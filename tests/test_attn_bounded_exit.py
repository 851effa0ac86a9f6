"""The attention kernels that give up on a bounded wait leave no copy in flight and no product
writing tensor memory that is freed, whichever role gives up, and nobody waits for a warp that
has left.  Read from the sources, as for the other kernels with bounded waits."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_decode_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["attn_few.cuh", "attn_many.cuh"])
def test_copies_are_drained_whatever_the_flag(name):
    text = source(name)
    drains = list(re.finditer(r"mbar_wait\(full\([^;]*50ull \* 1000 \* 1000\);", text))
    assert len(drains) == 1
    before = text[:drains[0].start()]
    last_copy = before.rfind("tma_load_")
    assert last_copy > 0 and "abort_flag" not in before[last_copy:]
    if name == "attn_many.cuh":
        assert re.search(r"if \(queries > 0\) mbar_wait\(q_full", text[drains[0].end():])


def test_tensor_memory_is_freed_behind_the_last_product():
    text = source("attn_many.cuh")
    teardown = text.rindex("mbar_wait(done, 0")
    assert teardown < text.index("tcgen05.dealloc")
    condition = text[text.rindex("if (", 0, teardown):teardown]
    assert "warp == 1" in condition and "abort_flag" not in condition


def test_the_computing_warps_leave_together():
    """Between a failed wait and the end of a segment the four warps agree on leaving."""
    text = source("attn_few.cuh")
    assert re.search(r"ok = all4\(ok\);\s*if \(!ok\) break;", text)
    waits = [m.start() for m in re.finditer(r"if \(!wait\(full", text)]
    assert len(waits) == 1 and text.index("ok = all4(ok);") > waits[0]


@pytest.mark.parametrize("name", ["attn_few.cuh", "attn_many.cuh"])
def test_every_wait_has_a_bound(name):
    text = source(name)
    assert "global_ns() - t0 > limit_ns" in text
    assert not re.search(r"while \(!mbar_(?:try|test)", text)


def test_the_registers_of_the_roles_fit_the_launch():
    text = source("attn_many.cuh")
    threads = int(re.search(r"kThreads = (\d+);", text).group(1))
    dec, inc = (int(re.search(r"setmaxnreg\.%s\.sync\.aligned\.u32 (\d+)" % w, text).group(1)) for w in ("dec", "inc"))
    launched = 65536 // threads // 8 * 8   # registers a thread at the launch, one block an SM
    assert 128 * dec + (threads - 128) * inc <= threads * launched


def test_a_stage_is_given_back_behind_a_fence():
    """Copies write a stage through another proxy than the matrix loads that read it."""
    text = source("attn_few.cuh")
    back = [m.start() for m in re.finditer(r"mbar_arrive\(empty\(", text)]
    assert len(back) == 1
    assert re.search(r"\n {12}fence_proxy_async\(\);\n {12}__syncwarp\(\);\n {12}if \(lane == 0\) $", text[:back[0]])
