"""The attention kernel for many rows hands registers from some of its warps to the others, and a
block with fewer than both shares need would wait for them without end: every instance is compiled
to have them, in the product and in the bounds-checking build, as the compiler reports it."""
import os
import re
import subprocess

import pytest

from gemm_decode_gb300 import build as q4build

THREADS, LOW, HIGH = 384, 88, 208   # 128 threads are left LOW registers, 256 get HIGH


@pytest.mark.parametrize("variant", sorted(q4build.VARIANTS))
def test_every_instance_has_the_registers_it_hands_over(variant, tmp_path):
    src = os.path.join(q4build.CSRC, "prefix_attn.cu")
    r = subprocess.run([q4build._nvcc(), *q4build.ARCH, *q4build.NVCC_FLAGS, *q4build.VARIANTS[variant][2], "-Xptxas", "-v",
                        "-c", src, "-o", str(tmp_path / "a.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    used = [int(m.group(1)) for m in re.finditer(
        r"Compiling entry function '[^']*attn_many_kernel[^']*'.*?Used (\d+) registers", r.stderr, re.S)]
    assert len(used) == 4   # two types, two head sizes
    assert all(n * THREADS >= 128 * LOW + (THREADS - 128) * HIGH for n in used), used


def test_the_launcher_refuses_a_kernel_with_fewer():
    """The shares that the kernel names, and that the launcher asks for, are the ones tested here."""
    with open(os.path.join(q4build.CSRC, "attn_many.cuh")) as f:
        text = f.read()
    assert re.findall(r"setmaxnreg\.(?:dec|inc)\.sync\.aligned\.u32 (\d+)", text) == [str(LOW), str(HIGH)]
    assert f"kRegisters = 128 * {LOW} + {THREADS - 128} * {HIGH};" in text and f"kThreads = {THREADS};" in text
