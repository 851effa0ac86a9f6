"""Beam selection and the reordering of pages against their definitions."""
import math

import decode_reference as ref
import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def step(torch, logits, scores, K, finished=None, eos=-1, **kw):
    groups, W = scores.shape
    V = logits.shape[1]
    new = lambda t: torch.full((groups, K), 77, device="cuda").to(t)  # noqa: E731
    tokens, parents, out, fin = new(torch.int32), new(torch.int32), new(torch.float32), new(torch.uint8)
    ws = torch.empty(q4.q4_beam_step_workspace(groups, W, K, V), device="cuda", dtype=torch.uint8)
    q4.q4_beam_step_run(logits, scores, tokens, parents, out, ws, finished=finished, out_finished=fin, eos=eos, **kw)
    torch.cuda.synchronize()
    return tokens, parents, out, fin


def check(torch, logits, scores, K, finished=None, eos=-1):
    got = step(torch, logits, scores, K, finished, eos)
    want = ref.beam_step(logits.cpu(), scores.cpu(), finished.cpu() if finished is not None else None, K, eos)
    # a sum of exponentials in binary32: each within 2^-21 (argument and function), sums of up to
    # V / 4096 + 24 steps; then binary64 and one rounding
    V = logits.shape[1]
    lost = 2.0 ** -21 + (V / 4096 + 24) * 2.0 ** -24
    fine = torch.isfinite(want[2])
    assert torch.equal(torch.isfinite(got[2].cpu()), fine)
    off = (got[2].cpu().double() - want[2])[fine].abs()
    assert (off <= lost + 2.0 ** -24 * want[2][fine].abs()).all()
    tokens, parents = got[0].cpu().long(), got[1].cpu().long()
    if not (torch.equal(tokens, want[0]) and torch.equal(parents, want[1])):
        same_but_for_close_scores(torch, tokens, parents, want, logits.cpu(), scores.cpu(), lost, eos)
    assert torch.equal(got[3].cpu() != 0, (tokens == eos) & (parents >= 0))
    return got


def same_but_for_close_scores(torch, tokens, parents, want, logits, scores, lost, eos):
    """Continuations of different beams whose exact scores are closer than the sums of
    exponentials are known may come in either order (rows that are permutations of one another
    have the same sum, and no order of additions makes that exact).  With every computed score
    within `lost` of the exact one, the j-th largest computed is within `lost` of the j-th
    largest exact, so the exact score of the j-th chosen is within 2 `lost` of it.  Within a beam
    the order is that of the logits, then the tokens, whatever the sums."""
    groups, W = scores.shape
    l = logits.double().reshape(groups, W, -1)
    for g in range(groups):
        seen = {}
        for j in range(tokens.shape[1]):
            v, w = int(tokens[g, j]), int(parents[g, j])
            assert (w < 0) == (want[1][g, j] < 0)
            if w < 0:
                continue
            exact = scores[g, w].double() + l[g, w, v] - torch.logsumexp(l[g, w], 0)
            assert abs(exact - want[2][g, j]) <= 2 * lost
            seen.setdefault(w, []).append(v)
        for w, vs in seen.items():
            assert torch.sort(l[g, w], descending=True, stable=True)[1][:len(vs)].tolist() == vs


@pytest.mark.parametrize("groups,W,K,V", [
    (1, 1, 1, 1), (1, 1, 1, 5), (1, 4, 4, 3), (3, 2, 5, 31), (2, 4, 4, 4095), (2, 4, 4, 4096), (2, 4, 8, 4097),
    (1, 4, 4, 151936), (5, 3, 3, 10007), (2, 32, 32, 1000), (1, 32, 32, 40001), (300, 2, 2, 130), (1, 2, 16, 300001)])
def test_beam_step_against_the_definition(torch, groups, W, K, V):
    torch.manual_seed(V + W)
    logits = 3 * torch.randn(groups * W, V, device="cuda")
    scores = -9 * torch.rand(groups, W, device="cuda")
    check(torch, logits, scores, K)
    done = (torch.rand(groups, W, device="cuda") < 0.4).to(torch.uint8)
    check(torch, logits, scores, K, done, V // 2)
    logits[torch.rand_like(logits) < 0.7] = -math.inf
    check(torch, logits, scores, K, None, 0)


def test_ties_go_to_the_lower_beam_then_the_lower_token(torch):
    V = 9000
    logits = torch.zeros(4, V, device="cuda")
    got = check(torch, logits, torch.zeros(1, 4, device="cuda"), 6)
    assert got[0].tolist() == [[0, 1, 2, 3, 4, 5]] and got[1].tolist() == [[0] * 6]
    logits[:, 7000:7004] = 2.0
    logits[:, 100] = 2.0
    got = check(torch, logits, torch.zeros(1, 4, device="cuda"), 7)
    assert got[0].tolist() == [[100, 7000, 7001, 7002, 7003, 100, 7000]]
    logits = torch.full((2, V), -3.4028234663852886e38, device="cuda")   # the lowest value: like any other
    check(torch, logits, torch.tensor([[-1.0, -2.0]], device="cuda"), 5)
    logits = torch.full((1, 10), 0.0, device="cuda")
    logits[0, 3] = -0.0   # both zeros are one value
    assert step(torch, logits, torch.zeros(1, 1, device="cuda"), 10)[0].tolist() == [list(range(10))]


def test_sorted_logits_and_many_candidates(torch):
    """Orders in which most logits pass the bound of their block."""
    for V in (4096, 8192, 20000):
        up = torch.arange(V, device="cuda").float() * 1e-3
        logits = torch.stack([up, up.flip(0), up.reshape(-1, 8).T.reshape(-1) if V % 8 == 0 else up, torch.zeros_like(up)])
        check(torch, logits, torch.zeros(1, 4, device="cuda"), 32)
        check(torch, logits, torch.zeros(4, 1, device="cuda"), 9)


def test_logits_that_are_not_finite(torch):
    V = 5000
    logits = torch.randn(4, V, device="cuda")
    logits[0, ::3] = math.nan
    logits[1, 1::2] = math.inf
    logits[2] = -math.inf
    logits[3] = math.nan
    scores = torch.tensor([[-1.0, -2.0, -0.1, -0.2]], device="cuda")
    check(torch, logits, scores, 8)
    got = check(torch, logits[2:], scores[:, 2:], 3)     # nothing to choose from
    assert got[0].tolist() == [[-1] * 3] and got[1].tolist() == [[-1] * 3] and got[3].tolist() == [[0] * 3]
    scores = torch.tensor([[-math.inf, 0.0, math.nan, math.inf]], device="cuda")   # the first step: one live beam
    logits = torch.randn(4, V, device="cuda")
    got = check(torch, logits, scores, 4)
    assert got[1].tolist() == [[1] * 4]
    check(torch, logits, scores, 4, torch.ones(1, 4, device="cuda", dtype=torch.uint8), 17)   # all finished


def test_rows_of_any_stride_and_alignment(torch):
    base = torch.randn(8 * 5003 + 3, device="cuda")
    scores = -torch.rand(2, 4, device="cuda")
    for lead, stride, V in ((0, 5000, 4999), (1, 5000, 5000), (0, 5003, 5000), (3, 5001, 4097)):
        check(torch, base[lead:lead + 8 * stride].as_strided((8, V), (stride, 1)), scores, 4)


def test_beam_step_is_the_same_every_time_and_in_a_graph(torch):
    logits, scores = torch.randn(8, 33333, device="cuda"), -torch.rand(2, 4, device="cuda")
    first = step(torch, logits, scores, 8)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step(torch, logits, scores, 8, flags=q4.Q4_RUN_OVERLAPPED)))
    tokens, parents = (torch.zeros(2, 8, device="cuda", dtype=torch.int32) for _ in range(2))
    out = torch.zeros(2, 8, device="cuda")
    ws = torch.empty(q4.q4_beam_step_workspace(2, 4, 8, 33333), device="cuda", dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_beam_step_run(logits, scores, tokens, parents, out, ws)
    logits.normal_()
    graph.replay()
    torch.cuda.synchronize()
    want = ref.beam_step(logits.cpu(), scores.cpu(), None, 8, -1)
    assert torch.equal(tokens.cpu().long(), want[0]) and torch.equal(parents.cpu().long(), want[1])


def setup(torch, groups, W, planes, heads, page, D, maxp, lens, t, layout="heads"):
    S = groups * W
    order = torch.randperm(2 * S + 3, device="cuda").to(torch.int32)
    lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
    tables = torch.randint(0, 2 * S, (S, maxp), device="cuda", dtype=torch.int32)
    at = (lens.long() // page).repeat_interleave(W)
    ok = at < maxp
    tables[torch.arange(S, device="cuda")[ok], at[ok]] = order[:S][ok]
    shape = (planes, 2 * S + 3, heads, page, D) if layout == "heads" else (2 * S + 3, page, planes, heads, D)
    pool = torch.randint(-100, 100, shape, device="cuda").to(t)
    if layout != "heads":
        pool = pool.permute(2, 0, 3, 1, 4)
    return lens, tables, order[S:2 * S].contiguous(), pool


@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("groups,W,planes,heads,page,D,maxp,t", [
    (1, 1, 2, 1, 16, 64, 4, "bfloat16"), (1, 4, 48, 2, 16, 64, 16, "bfloat16"), (3, 3, 5, 3, 7, 9, 3, "float16"),
    (2, 8, 4, 8, 32, 128, 5, "float16"), (5, 2, 1, 1, 1, 2, 9, "float32"), (1, 300, 2, 1, 16, 8, 2, "bfloat16"),
    (2, 2, 3, 2, 64, 4, 1, "float8_e4m3fn")])
def test_reorder_against_the_definition(torch, layout, groups, W, planes, heads, page, D, maxp, t):
    torch.manual_seed(W + D)
    for last in range(4):
        # no token, a full last page, within a page, everything full
        n = [[0, page * (maxp - 1), page * maxp - 1, page * maxp][(g + last) % 4] for g in range(groups)]
        if last == 3:
            n = [int(v) for v in torch.randint(0, maxp * page, (groups,))]
        lens, tables, spare, pool = setup(torch, groups, W, planes, heads, page, D, maxp, n, getattr(torch, t), layout)
        parents = torch.randint(0, W, (groups, W), device="cuda", dtype=torch.int32)
        parents[:, 0] = W - 1
        if last == 2:
            parents[0, -1] = -1   # counts as itself
        new, left = torch.full_like(tables, -7), torch.full_like(spare, -7)
        want = ref.reorder(tables.cpu(), lens.cpu(), parents.cpu(), spare.cpu(), pool.cpu().float())
        q4.q4_beam_reorder_run(tables, lens, parents, spare, new, left, pool)
        torch.cuda.synchronize()
        assert torch.equal(new.cpu(), want[0]) and torch.equal(left.cpu(), want[1])
        assert torch.equal(pool.cpu().float(), want[2])


def test_reorder_leaves_pages_outside_the_pool_alone(torch):
    lens, tables, spare, pool = setup(torch, 1, 3, 2, 1, 16, 8, 4, [20], torch.bfloat16)
    parents = torch.tensor([[1, 2, 0]], device="cuda", dtype=torch.int32)
    tables[2, 1] = pool.shape[1]    # sequence 1's parent
    spare[2] = -1
    new, left = torch.zeros_like(tables), torch.zeros_like(spare)
    want = ref.reorder(tables.cpu(), lens.cpu(), parents.cpu(), spare.cpu(), pool.cpu())
    q4.q4_beam_reorder_run(tables, lens, parents, spare, new, left, pool)
    torch.cuda.synchronize()
    assert torch.equal(new.cpu(), want[0]) and torch.equal(left.cpu(), want[1]) and torch.equal(pool.cpu(), want[2])
