"""Attention at sizes where the plan, the division of the work and the joining take other ways:
tables of the most tokens, many groups, many runs, many segments and many parts."""
import math

import decode_reference as ref
import pytest
import test_gpu_prefix_attn as attn
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


@pytest.mark.parametrize("kind", ["own", "shared", "both"])
def test_tables_of_the_most_tokens(torch, kind):
    """Just below 2^31 keys.  Keys are zeros, so every weight is 1 and the output is the sum of the
    values by their number; pages outside the pool are zeros, so few values count.

    Sums of ones are exact up to 2^24, as much as a CTA's share is; then 15 additions of parts at most,
    in binary32, and a logarithm to base 2 with its factor."""
    page, D, columns = 16, 64, 2 ** 27 - 1
    n = columns * page
    assert n == 2 ** 31 - 16
    kc = torch.zeros(3, 1, page, D, device="cuda", dtype=torch.bfloat16)
    vc = torch.randn(3, 1, page, D, device="cuda").to(torch.bfloat16)
    table = torch.full((1, columns), -1, device="cuda", dtype=torch.int32)
    for i, at in enumerate((0, 5, columns // 2, columns - 2, columns - 1)):
        table[0, at] = i % 3
    lens = torch.full((1,), 2 ** 31 - 1, device="cuda", dtype=torch.int32)   # (clamped to the table)
    S = 17 if kind == "shared" else 1
    p = dict(q=torch.randn(S, 1, D, device="cuda").to(torch.bfloat16), k_cache=kc, v_cache=vc, group_offsets=None,
             shared_pages=None, shared_lens=None, limits=None, own_pages=None, own_lens=None)
    if kind != "own":
        p["shared_pages"], p["shared_lens"] = table, lens
    if kind != "shared":
        p["own_pages"], p["own_lens"] = table, lens
    out, lse = attn.run(torch, p, out_dtype=torch.float32)
    assert q4.q4gemv_device_status() == q4.Q4_OK
    v = vc[torch.tensor([0, 1, 2, 0, 1], device="cuda")].double().cpu()
    times = 2 if kind == "both" else 1
    want = (v.sum((0, 1, 2)) / n).expand(S, 1, D)   # (both: twice the values by twice the keys)
    steps = 15 * 2.0 ** -24
    ref.within(out, want, (v.abs().sum((0, 1, 2)) / n * (2 * steps + 80 * 2.0 ** -24)).expand(S, 1, D), "out")
    log = torch.full((S, 1), math.log(n * times), dtype=torch.float64)
    ref.within(lse, log, steps + 4 * 2.0 ** -24 * log, "lse")


def test_a_refused_call_launches_nothing(torch):
    """Rows of queries too far apart for a tensor map are refused before the plan is written."""
    p = attn.problem(torch, [20], [40], None, 8, 2, 64, 16, torch.bfloat16)
    S, Hq, D = p["q"].shape
    ws = torch.full((q4.q4_prefix_attn_workspace(S, 1, Hq, 2, D),), 255, device="cuda", dtype=torch.uint8)
    out = torch.full((S, Hq, D), 9.0, device="cuda", dtype=torch.bfloat16)
    far = 1 << 50   # an address that nothing else of the call is near; never read
    cache = q4._cache(0, p["k_cache"], p["v_cache"])
    a = q4._ATTN.pack(S, Hq, 1, q4.Q4_BF16, p["shared_pages"].shape[1], 0, 0.1, far, 2 ** 39, *cache, 0,
                      p["shared_pages"].data_ptr(), p["shared_lens"].data_ptr(), 0, 0, 0, out.data_ptr(), 0, ws.data_ptr(),
                      ws.numel())
    assert q4.lib().q4_prefix_attn_run(a, None, None) == q4.Q4_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (ws == 255).all() and (out == 9).all()
    check = attn.check(torch, p, ws=ws)   # and the call after it is right
    assert torch.isfinite(check[0]).all()
