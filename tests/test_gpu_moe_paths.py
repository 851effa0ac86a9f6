"""The expert products on paths that depend on how the work is divided: waits that run out
while copies are under way, and so on.  GPU parity against the plain 64-bit forms of
moe_reference.py.
"""
import moe_reference as ref
import numpy as np
import pytest
from gpu_util import torch_cuda
from test_gpu_moe import groups, make_weights, num, run_experts, to, within, work

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


@pytest.mark.parametrize("bf16,T", [(False, 4), (True, 4), (True, 80)])
@pytest.mark.parametrize("K", [128, 256, 384])
def test_products_that_give_up_at_once_leave_the_next_ones_alone(torch, bf16, T, K):
    """Items of one to three units: all copies of a CTA are under way when its waits run out.
    The products launched behind them give their values and report nothing."""
    rng = np.random.default_rng(K + T)
    E, N = 3, 520
    t = torch.bfloat16 if bf16 else torch.float32
    weights = make_weights(rng, E, N, K, 32, False)
    offsets, rows = groups(rng, E, 1, T, "even")
    x = num(torch.from_numpy(rng.normal(0, 1, (T, K))).to(t))
    args = [to(torch, a) for a in weights] + [to(torch, x, t), to(torch, rows), to(torch, offsets)]
    y, z = (torch.zeros(T, N, dtype=t, device="cuda") for _ in range(2))
    ws = work(torch, q4.q4moe_gemm_workspace(T, T, N, K, E, t))
    want, bound = ref.experts(ref.dequant(*weights, 32), x, rows, offsets, np.zeros((T, N)), False, bf16)
    for _ in range(8):
        q4.q4moe_gemm_run(*args, z, ws, group=32, wait_timeout_ns=0)
        q4.q4moe_gemm_run(*args, y, ws, group=32)
    torch.cuda.synchronize()
    assert q4.q4gemv_device_status() in (q4.Q4_OK, q4.Q4_ERR_TIMEOUT)
    assert q4.q4gemv_device_status() == q4.Q4_OK
    within(num(y), want, bound, "behind a product that gave up")
    y.zero_()
    q4.q4moe_gemm_run(*args, y, ws, group=32)
    torch.cuda.synchronize()
    assert q4.q4gemv_device_status() == q4.Q4_OK
    within(num(y), want, bound, "after")
