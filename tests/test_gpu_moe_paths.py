"""The expert products on paths that depend on how the work is divided: waits that run out
while copies are under way, items whose K several CTAs share, rows of scales longer than one
chunk.  GPU parity against plain 64-bit forms (moe_reference.py, moe_bounds.py).
"""
import os
import re

import moe_bounds as mb
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


# ---------------------------------------------------------------- items shared by several CTAs

def k_join():
    """Units that the plan takes a join of partial sums to cost."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_decode_gb300", "csrc",
                        "moe_gemm_common.cuh")
    with open(path) as f:
        return int(re.search(r"kJoin = (\d+);", f.read()).group(1))


def division(counts, N, K, g, bf16, sms):
    """(rows of x per item, whether CTAs share the units of an item) of a call whose experts
    have counts[e] rows: the rules of the kernels, worked out on the host."""
    R, E = sum(counts), len(counts)
    if bf16:
        rt, nt = (1, 32) if R <= 24 * E else (2, 128)
    elif g == 32 or R <= 8 * E:
        rt, nt = 1, 16
    else:
        rt, nt = 1, 32 if g == 64 or R <= 24 * E else 64
    items = sum(-(-c // nt) for c in counts) * -(-N // (128 * rt))
    units, waves = -(-K // 128), -(-items // sms)
    return nt, not (waves >= 16 or waves * sms * units <= items * units + k_join() * sms)


def shared_call(torch, counts, N, K, g, sym, swiglu, bf16, gather, seed=0):
    """A call over random weights whose items the CTAs share, as a function, and its values."""
    rng = np.random.default_rng(seed + K + N)
    E, R = len(counts), sum(counts)
    t = torch.bfloat16 if bf16 else torch.float32
    weights = make_weights(rng, E, N, K, g, sym)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    Tx = R // 2 + 1 if gather else R
    rows = rng.integers(0, Tx, R).astype(np.int32) if gather else None
    x = num(torch.from_numpy(rng.normal(0, 1, (Tx, K))).to(t))
    y = torch.full((R, N // 2 if swiglu else N), 7.0, dtype=t, device="cuda")
    args = [to(torch, a) for a in weights] + [to(torch, x, t), to(torch, rows), to(torch, offsets), y,
                                               work(torch, q4.q4moe_gemm_workspace(R, Tx, N, K, E, t))]

    def call(**kw):
        q4.q4moe_gemm_run(*args, group=g, epilogue=q4.Q4_EPILOGUE_SWIGLU if swiglu else q4.Q4_EPILOGUE_NONE, **kw)
        return y
    want, bound = mb.experts(ref.dequant(*weights, g), x, rows, offsets, np.full(tuple(y.shape), 7.0), swiglu, bf16, g)
    return call, want, bound, weights, x, rows, offsets


# counts of rows per expert, N, K, g, type, rows of x per item: every instance of the two
# kernels, items that start and end inside a CTA's share, items over many CTAs, partial tiles
# of weights and of x, and K whose last unit has 32, 64, 96 or 128 elements
SHARED = [
    ([60, 131, 5], 700, 6400, 64, True, 128),
    ([100, 40], 512, 4864, 128, True, 128),
    ([33, 0, 129], 260, 6432, 32, True, 128),
    ([70], 1030, 6496, 32, True, 128),
    ([200, 3], 300, 4928, 64, True, 128),
    ([9, 3, 0, 20], 390, 4864, 32, True, 32),
    ([24], 140, 14336, 128, True, 32),
    ([17, 1, 6], 258, 4928, 64, True, 32),
    ([5, 0, 11], 390, 4864, 32, False, 16),
    ([8, 3], 130, 6496, 32, False, 16),
    ([7], 514, 14336, 128, False, 16),
    ([40, 20], 300, 4864, 64, False, 32),
    ([20, 12], 516, 6400, 128, False, 32),
    ([65, 30, 1], 260, 4864, 128, False, 64),
    ([130], 516, 6400, 128, False, 64),
]


@pytest.mark.parametrize("counts,N,K,g,bf16,nt", SHARED)
def test_items_shared_by_several_ctas(torch, counts, N, K, g, bf16, nt):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert division(counts, N, K, g, bf16, sms) == (nt, True)
    for sym, swiglu, gather in ((False, False, True), (True, True, False)):
        call, want, bound, *_ = shared_call(torch, counts, N, K, g, sym, swiglu, bf16, gather)
        first = call().clone()
        within(num(first), want, bound, f"sym {sym}")
        for _ in range(4):   # whoever arrives last, bit for bit
            assert torch.equal(call(flags=q4.Q4_RUN_OVERLAPPED), first)
    assert q4.q4gemv_device_status() == q4.Q4_OK


@pytest.mark.parametrize("counts,N,K,g,bf16,nt", [SHARED[0], SHARED[5], SHARED[8], SHARED[13]])
def test_shared_items_in_a_graph(torch, counts, N, K, g, bf16, nt):
    """Captured with one division of the rows, replayed with others."""
    call, _, _, weights, x, rows, offsets = shared_call(torch, counts, N, K, g, False, False, bf16, False)
    E, R = len(counts), sum(counts)
    t = torch.bfloat16 if bf16 else torch.float32
    W = ref.dequant(*weights, g)
    ot, y = to(torch, offsets), torch.zeros(R, N, dtype=t, device="cuda")
    args = [to(torch, a) for a in weights] + [to(torch, x, t), None, ot, y,
                                              work(torch, q4.q4moe_gemm_workspace(R, R, N, K, E, t))]
    q4.q4moe_gemm_run(*args, group=g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4moe_gemm_run(*args, group=g)
    for o in (offsets, np.minimum(offsets, R // 3), np.where(np.arange(E + 1) == 0, 0, R).astype(np.int32)):
        ot.copy_(to(torch, o))
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want, bound = mb.experts(W, x, None, o, np.full((R, N), 7.0), False, bf16, g)
        within(num(y), want, bound, str(o.tolist()))


@pytest.mark.parametrize("counts,N,K,g,bf16,nt", [SHARED[1], SHARED[6], SHARED[10], SHARED[11], SHARED[14]])
def test_giving_up_with_shared_items(torch, counts, N, K, g, bf16, nt):
    """A zero bound is reported once, and the next call has its values."""
    call, want, bound, *_ = shared_call(torch, counts, N, K, g, True, False, bf16, False)
    call(wait_timeout_ns=0)
    torch.cuda.synchronize()
    assert q4.q4gemv_device_status() == q4.Q4_ERR_TIMEOUT
    assert q4.q4gemv_device_status() == q4.Q4_OK
    within(num(call()), want, bound, "after the timeout")
    assert q4.q4gemv_device_status() == q4.Q4_OK


# ---------------------------------------------------------------- many rows per expert

@pytest.mark.parametrize("K,g", [(640, 32), (1056, 32), (1120, 32), (2112, 64), (2880, 64), (2304, 128)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_rows_with_several_chunks_of_scales(torch, K, g, swiglu):
    """More than 16 groups in a row (18 to 45), the last unit of K of 32, 64, 96 or 128 elements."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    counts = [130, 2, 0, 71]
    assert division(counts, 300, K, g, True, sms) == (128, False)
    for sym, gather in ((False, True), (True, False)):
        call, want, bound, *_ = shared_call(torch, counts, 300, K, g, sym, swiglu, True, gather)
        within(num(call()), want, bound, f"sym {sym}")
