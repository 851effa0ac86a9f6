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


def ragged(n, most):
    """Sizes of n groups, 0 to `most`, empty ones side by side and at both ends."""
    return [0, 0] + [(7 * g + g // 5) % (most + 1) for g in range(n - 4)] + [0, 0]


def with_limits(torch, p, kind):
    if kind == "limits":
        S = p["q"].shape[0]
        limits = torch.randint(-2, 70, (S,), device="cuda")
        limits[::17] = 0
        p["limits"] = limits.to(torch.int32)
    return p


# groups in one warp's lanes up to 31, in shared memory up to 1024, in the workspace beyond
GROUPS = [(31, 20, 4, 2), (32, 20, 4, 2), (33, 3, 4, 2), (130, 9, 4, 2), (1023, 3, 8, 1), (1024, 3, 8, 1), (1025, 3, 8, 1),
          (2050, 3, 16, 1)]   # (no more groups than queries: others are refused)


@pytest.mark.parametrize("kind", ["plain", "limits"])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("groups,most,Hq,Hkv", GROUPS)
def test_numbers_of_groups(torch, groups, most, Hq, Hkv, own, kind):
    sizes = ragged(groups, most)
    S = sum(sizes)
    shared = [(11 * g) % 67 for g in range(groups)]
    p = attn.problem(torch, sizes, shared, [(5 * s) % 23 for s in range(S)] if own else None, Hq, Hkv, 64, 16,
                     torch.bfloat16, stale=groups < 200)
    attn.check(torch, with_limits(torch, p, kind))


@pytest.mark.parametrize("kind", ["plain", "limits"])
@pytest.mark.parametrize("sizes,own", [([2100], False), ([2100], True), ([3] * 700, False), ([3, 0, 5, 1] * 250, True)])
def test_numbers_of_runs(torch, sizes, own, kind):
    """Two queries a run (128 query heads of a kv head): more runs than shared memory holds."""
    S = sum(sizes)
    p = attn.problem(torch, sizes, [40 + g % 30 for g in range(len(sizes))], [s % 9 for s in range(S)] if own else None,
                     128, 1, 64, 16, torch.float16, stale=False)
    attn.check(torch, with_limits(torch, p, kind))


def test_many_segments_a_cta(torch):
    """More than the 32 entries that a CTA holds in shared memory, in both kernels."""
    S = 12000
    p = attn.problem(torch, [S], None, [1 + (13 * s) % 40 for s in range(S)], 1, 1, 64, 16, torch.bfloat16, stale=False)
    attn.check(torch, p)
    S = 6000
    p = attn.problem(torch, [1] * S, [1 + (29 * s) % 90 for s in range(S)], None, 32, 1, 64, 16, torch.bfloat16, stale=False)
    attn.check(torch, p)
    attn.check(torch, with_limits(torch, p, "limits"))


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 64), (14, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("queries", [1, 3, 20, 90])
def test_rows_of_many_parts(torch, queries, Hq, Hkv, D):
    """A long segment is shared by all CTAs: a row has parts by the hundred, joined 32 at a time."""
    n = 30011
    one = attn.problem(torch, [queries], [n], None, Hq, Hkv, D, 64, torch.bfloat16)
    attn.check(torch, one)                                                   # shared segments alone
    one["limits"] = torch.linspace(1, n, queries, device="cuda").to(torch.int32)
    attn.check(torch, one)
    attn.check(torch, attn.problem(torch, [queries], [n], [9000 + s for s in range(min(queries, 3))] + [3] * (queries - min(queries, 3)),
                                   Hq, Hkv, D, 64, torch.float16))           # both kinds
    if queries <= 3:
        attn.check(torch, attn.problem(torch, [queries], None, [n - s for s in range(queries)], Hq, Hkv, D, 64, torch.bfloat16))


def test_waits_of_any_bound_end(torch):
    """Whatever a wait's bound, the call ends: with the right result, or with a status that says
    that a wait gave up, after which a call in the same workspace is right."""
    for case in (dict(sizes=[70, 2], shared=[3000, 500], own=[200] * 72), dict(sizes=[300], shared=[700], own=None),
                 dict(sizes=[6], shared=None, own=[5000] * 6)):
        p = attn.problem(torch, case["sizes"], case["shared"], case["own"], 8, 2, 128, 16, torch.bfloat16)
        S, groups = p["q"].shape[0], len(case["shared"] or [])
        ws = torch.empty(q4.q4_prefix_attn_workspace(S, groups, 8, 2, 128), device="cuda", dtype=torch.uint8)
        right, lse = attn.check(torch, p, ws=ws)
        ended = set()
        for bound in (0, 1, 100, 1000, 3000, 10000, 10 ** 9):
            out, l = attn.run(torch, p, ws=ws, wait_timeout_ns=bound)
            status = q4.q4gemv_device_status()
            assert status in (q4.Q4_OK, q4.Q4_ERR_TIMEOUT)
            ended.add(status)
            if status == q4.Q4_OK:
                assert torch.equal(out, right) and torch.equal(l, lse)
            out, l = attn.run(torch, p, ws=ws)
            assert q4.q4gemv_device_status() == q4.Q4_OK and torch.equal(out, right) and torch.equal(l, lse)
        assert ended == {q4.Q4_OK, q4.Q4_ERR_TIMEOUT}
