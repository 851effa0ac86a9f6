"""Attention over a shared and an own segment against the formula in 64 bits."""
import math

import decode_reference as ref
import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def problem(torch, sizes, shared, own, Hq, Hkv, D, page, t16, layout="heads", stale=True, qmul=1.5, seed=0, extra=0):
    """Groups of these sizes with these shared lengths (None: no shared segments), own lengths per
    query (None: none).  Behind every sequence's last token the pages hold NaN and infinities."""
    torch.manual_seed(sum(sizes) * 7 + D + page + seed)
    S = sum(sizes) + extra
    seqs = list(shared or []) + list(own or [])
    need = [(n + page - 1) // page for n in seqs]
    pages = sum(need) + 2
    shape = (pages, Hkv, page, D)
    if layout == "heads":
        kc, vc = (torch.randn(shape, device="cuda").to(t16) for _ in range(2))
    elif layout == "tokens":
        kc, vc = (torch.randn(pages, page, Hkv, D, device="cuda").to(t16).transpose(1, 2) for _ in range(2))
    else:
        both = torch.randn(pages, 2, Hkv, page, D, device="cuda").to(t16)
        kc, vc = both[:, 0], both[:, 1]
    free = torch.randperm(pages, device="cuda").to(torch.int32)
    at, tables = 0, []
    for n, m in zip(seqs, need):
        tables.append(free[at:at + m])
        if stale and n % page:
            p = int(free[at + m - 1])
            kc[p, :, n % page:] = float("nan")
            vc[p, :, n % page:] = float("inf")
            vc[p, :, n % page::2] = float("nan")
        at += m
    if stale:
        for p in free[at:].tolist():
            kc[p], vc[p] = float("nan"), float("nan")

    def table(rows, width):
        t = torch.full((len(rows), width), -5, device="cuda", dtype=torch.int32)
        for i, r in enumerate(rows):
            t[i, :len(r)] = r
        return t

    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    p = dict(q=(qmul * torch.randn(S, Hq, D, device="cuda")).to(t16), k_cache=kc, v_cache=vc, group_offsets=None,
             shared_pages=None, shared_lens=None, limits=None, own_pages=None, own_lens=None)
    if shared is not None:
        offsets = [0]
        for n in sizes:
            offsets.append(offsets[-1] + n)
        p["group_offsets"] = i32(offsets)
        p["shared_pages"] = table(tables[:len(shared)], max(1, max(need[:len(shared)])) + 1)
        p["shared_lens"] = i32(shared)
    if own is not None:
        k = len(shared or [])
        p["own_pages"] = table(tables[k:], max(1, max(need[k:])) + 2)
        p["own_lens"] = i32(own)
    return p


def run(torch, p, out_dtype=None, scale=None, ws=None, **kw):
    S, Hq, D = p["q"].shape
    groups = p["shared_lens"].numel() if p["shared_lens"] is not None else 0
    out = torch.full((S, Hq, D), 9.0, device="cuda", dtype=out_dtype or p["q"].dtype)
    lse = torch.full((S, Hq), 9.0, device="cuda")
    if ws is None:
        ws = torch.empty(q4.q4_prefix_attn_workspace(S, groups, Hq, p["k_cache"].shape[1], D), device="cuda",
                         dtype=torch.uint8)
        ws.fill_(255)   # its contents mean nothing: NaN here
    q4.q4_prefix_attn_run(p["q"], p["k_cache"], p["v_cache"], out, ws, lse=lse, scale=scale,
                          **{n: p[n] for n in ("group_offsets", "shared_pages", "shared_lens", "limits", "own_pages",
                                               "own_lens")}, **kw)
    return out, lse


def check(torch, p, out_dtype=None, scale=None, **kw):
    out, lse = run(torch, p, out_dtype, scale, **kw)
    assert q4.q4gemv_device_status() == q4.Q4_OK
    cpu = {n: (v.cpu() if v is not None else None) for n, v in p.items()}
    t16 = p["q"].dtype
    s = p["q"].shape[2] ** -0.5 if scale is None else scale
    o, l, bo, bl = ref.attention(cpu["q"], cpu["k_cache"], cpu["v_cache"], cpu["group_offsets"], cpu["shared_pages"],
                                 cpu["shared_lens"], cpu["limits"], cpu["own_pages"], cpu["own_lens"], s, t16)
    ref.within(out, o, (1 + 2.0 ** -7) * bo + ref.rounding(o, out.dtype), "out")
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse.cpu()) & (lse.cpu() < 0), empty)
    ref.within(lse.cpu()[~empty], l[~empty], bl[~empty], "lse")
    return out, lse


# (group sizes, shared lengths, own lengths per query, Hq, Hkv, D, page)
CASES = [
    ([1], [1], None, 1, 1, 64, 16),
    ([1], None, [1], 1, 1, 128, 16),
    ([1], None, [777], 8, 2, 128, 16),
    ([4], [1000], [20, 1, 0, 33], 32, 8, 128, 16),
    ([4], [16], [16, 32, 48, 64], 14, 2, 64, 16),
    ([3, 1, 8], [300, 0, 65], [5, 0, 0, 0, 64, 65, 63, 1, 200, 17, 128, 129], 28, 4, 128, 32),
    ([5, 0, 2], [40, 50, 129], None, 6, 2, 64, 64),
    ([33], [257], [3] * 33, 8, 8, 64, 128),
    ([70], [640], [0] * 69 + [400], 8, 2, 128, 16),
    ([40], [1300], None, 16, 2, 128, 64),
    ([150], [513], [7] * 150, 5, 1, 64, 16),
    ([9], [500], [100] * 9, 64, 1, 128, 32),
    ([2], [200], [130, 5], 128, 1, 64, 32),
    ([1, 2, 3, 4, 5, 6, 7, 8], [1, 15, 16, 17, 127, 128, 129, 1], [i * 3 for i in range(36)], 9, 3, 128, 16),
    ([20], None, [64 * i for i in range(20)], 32, 8, 64, 256),
]


@pytest.mark.parametrize("t16", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_against_the_formula(torch, case, t16):
    sizes, shared, own, Hq, Hkv, D, page = CASES[case]
    p = problem(torch, sizes, shared, own, Hq, Hkv, D, page, getattr(torch, t16))
    check(torch, p)
    check(torch, p, out_dtype=torch.float32, scale=0.31)


@pytest.mark.parametrize("layout", ["heads", "tokens", "paired"])
@pytest.mark.parametrize("page", [16, 64, 512])
def test_layouts_of_the_pools(torch, layout, page):
    p = problem(torch, [30, 3], [400, 90], [11] * 33, 8, 2, 128, page, torch.bfloat16, layout)
    check(torch, p)
    # queries as a part of wider rows
    wide = torch.randn(33, 12, 128, device="cuda").bfloat16()
    p["q"] = wide[:, 2:10]
    check(torch, p)


@pytest.mark.parametrize("n,before,Hq,Hkv,D,page", [(1, 0, 4, 4, 64, 16), (200, 0, 8, 2, 128, 16), (77, 50, 14, 2, 64, 32),
                                                    (130, 400, 7, 1, 128, 64), (300, 1, 2, 2, 64, 128)])
def test_causal_prompt(torch, n, before, Hq, Hkv, D, page):
    """The last n tokens of a prompt, each seeing the tokens before it and itself."""
    p = problem(torch, [n], [n + before], None, Hq, Hkv, D, page, torch.bfloat16)
    p["limits"] = (before + 1 + torch.arange(n, device="cuda")).to(torch.int32)
    check(torch, p)


def test_limits_of_any_kind(torch):
    """Padding queries without a key, limits beyond the segment, in no order; two prompts."""
    p = problem(torch, [60, 41], [333, 100], None, 8, 2, 128, 16, torch.float16)
    limits = torch.randint(-3, 400, (101,), device="cuda")
    limits[:5], limits[20:58], limits[70] = 0, 0, -2 ** 31
    limits[59] = 2 ** 31 - 1
    p["limits"] = limits.to(torch.int32)
    out, lse = check(torch, p)
    assert (out[:5] == 0).all() and torch.isinf(lse[:5]).all()
    p = problem(torch, [60, 41], [333, 100], [9] * 101, 8, 2, 128, 16, torch.float16)
    p["limits"] = limits.to(torch.int32)
    check(torch, p)


def test_queries_without_a_key_give_zeros(torch):
    p = problem(torch, [3], [0], [0, 0, 4], 4, 2, 64, 16, torch.bfloat16)
    out, lse = check(torch, p)
    assert (out[:2] == 0).all()
    p = problem(torch, [20], [0], None, 8, 2, 128, 16, torch.bfloat16)
    out, lse = check(torch, p)
    assert (out == 0).all() and torch.isinf(lse).all()


def test_queries_that_no_group_has(torch):
    """They see their own segment alone."""
    p = problem(torch, [20], [200], [5] * 27, 8, 2, 128, 16, torch.bfloat16, extra=7)
    check(torch, p)
    p["group_offsets"] = torch.tensor([3, 21], device="cuda", dtype=torch.int32)
    check(torch, p)
    p["own_pages"] = p["own_lens"] = None
    out, _ = check(torch, p)
    assert (out[:3] == 0).all() and (out[21:] == 0).all()


def test_contents_that_make_no_sense_stay_in_bounds(torch):
    """Lengths beyond the tables, page ids outside the pool (zeros), offsets in no order."""
    p = problem(torch, [4, 20, 6], [90, 200, 33], [12] * 30, 8, 2, 128, 16, torch.bfloat16, stale=False)
    p["shared_pages"][1, 2], p["shared_pages"][0, 0], p["own_pages"][4, 0] = -1, 2 ** 31 - 1, p["k_cache"].shape[0]
    check(torch, p)
    p["shared_lens"][1], p["own_lens"][3], p["own_lens"][4] = 2 ** 31 - 1, 10 ** 6, -4
    check(torch, p)
    p["group_offsets"] = torch.tensor([5, 2, 900, -4], device="cuda", dtype=torch.int32)
    check(torch, p)
    p["group_offsets"] = torch.tensor([-2, -1, 4, 9], device="cuda", dtype=torch.int32)
    check(torch, p)


def test_scores_far_apart_and_not_finite(torch):
    """Large scores of both signs, keys that grow so that the maximum keeps moving, a query that is NaN."""
    for t16 in (torch.bfloat16, torch.float16):
        p = problem(torch, [30], [700], [65] * 30, 8, 2, 128, 16, t16, qmul=12.0)
        check(torch, p)
        p = problem(torch, [30], [600], [40] * 30, 8, 2, 128, 16, t16, stale=False)
        pages = p["shared_pages"][0][:38].long()
        grow = torch.linspace(0, 1, 38, device="cuda")[:, None, None, None]
        p["k_cache"][pages] = (p["k_cache"][pages].float() * grow * 4).to(t16)
        check(torch, p)
        check(torch, p, scale=-0.5)
        check(torch, p, scale=0.0)
    p["q"][3, 2] = float("nan")
    out, lse = run(torch, p)
    assert torch.isnan(out[3, 2]).all() and torch.isnan(lse[3, 2])
    good = torch.ones(30, 8, dtype=torch.bool)
    good[3, 2] = False
    assert torch.isfinite(out.cpu()[good]).all()


def test_a_sequence_of_equal_keys_averages_its_values(torch):
    """Weights are equal: the output is the mean of the values, over a length that splits."""
    n = 3000
    p = problem(torch, [20], [n], None, 8, 2, 64, 16, torch.float16, stale=False)
    p["k_cache"].fill_(1.0)
    out, lse = check(torch, p)
    x = p["q"].double().sum(2).cpu() / 8
    assert torch.allclose(lse.double().cpu(), x + math.log(n), rtol=0, atol=1e-4)


def test_the_same_every_time_and_on_another_stream(torch):
    p = problem(torch, [40], [5000], [300] * 40, 8, 2, 128, 16, torch.bfloat16)
    a, la = run(torch, p)
    for _ in range(3):
        b, lb = run(torch, p, flags=q4.Q4_RUN_OVERLAPPED)
        assert torch.equal(a, b) and torch.equal(la, lb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    r = problem(torch, [7], [900], [30] * 7, 8, 2, 128, 16, torch.bfloat16, seed=3)
    c, _ = run(torch, r)
    torch.cuda.synchronize()
    for _ in range(5):   # two calls at once, a workspace each
        with torch.cuda.stream(s1):
            x, _ = run(torch, p)
        with torch.cuda.stream(s2):
            y, _ = run(torch, r)
        torch.cuda.synchronize()
        assert torch.equal(x, a) and torch.equal(y, c)


def test_captured_once_and_replayed_as_the_sequences_grow(torch):
    S, page = 12, 16
    p = problem(torch, [6, 6], [200, 100], [150] * S, 8, 2, 128, page, torch.bfloat16, stale=False)
    ws = torch.empty(q4.q4_prefix_attn_workspace(S, 2, 8, 2, 128), device="cuda", dtype=torch.uint8)
    run(torch, p, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run(torch, p, ws=ws)
    for n, m in ((0, 1), (1, 0), (17, 200), (150, 64)):
        p["own_lens"].fill_(n)
        p["own_lens"][3] = 150 - n
        p["shared_lens"][0] = m
        p["q"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        again, lagain = check(torch, p)
        assert torch.equal(out, again) and torch.equal(lse, lagain)


def test_a_cache_beyond_32_bits(torch):
    """Pages whose elements lie more than 2^32 elements into the pool, and a long sequence over them."""
    pages, page, D = 2 ** 32 // (2 * 64 * 64) + 40, 64, 64
    kc = torch.zeros(pages, 2, page, D, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    n = 36 * page - 7
    table = torch.arange(pages - 36, pages, device="cuda", dtype=torch.int32)[None]
    kc[pages - 36:].normal_()
    vc[pages - 36:].normal_()
    p = dict(q=torch.randn(20, 4, D, device="cuda").bfloat16(), k_cache=kc, v_cache=vc, group_offsets=None,
             shared_pages=table, shared_lens=torch.tensor([n], device="cuda", dtype=torch.int32), limits=None,
             own_pages=table.repeat(20, 1), own_lens=torch.full((20,), 100, device="cuda", dtype=torch.int32))
    out, lse = run(torch, p)
    k, v = (c[pages - 36:].cpu() for c in (kc, vc))
    small = {"shared_pages": table.cpu() - (pages - 36), "own_pages": table.cpu().repeat(20, 1) - (pages - 36)}
    o, l, bo, bl = ref.attention(p["q"].cpu(), k, v, None, small["shared_pages"], p["shared_lens"].cpu(), None,
                                 small["own_pages"], p["own_lens"].cpu(), D ** -0.5, torch.bfloat16)
    ref.within(out, o, 1.01 * bo + ref.rounding(o, torch.bfloat16), "out")
    ref.within(lse, l, bl, "lse")


def test_bounded_waits_report_a_timeout_and_the_next_call_is_right(torch):
    """A bound of 0: each wait that is not satisfied at once gives up, the kernels end, and the
    status says so.  (Groups of both kinds: both kernels.)"""
    p = problem(torch, [70, 2], [3000, 500], [200] * 72, 8, 2, 128, 16, torch.bfloat16)
    run(torch, p, wait_timeout_ns=0)
    assert q4.q4gemv_device_status() == q4.Q4_ERR_TIMEOUT
    assert q4.q4gemv_device_status() == q4.Q4_OK
    check(torch, p)


def test_a_prompt_and_a_search_in_one_workspace(torch):
    """Calls of other sizes and kinds one after another in the largest one's workspace."""
    a = problem(torch, [300], [300], None, 8, 2, 128, 16, torch.bfloat16)
    a["limits"] = (1 + torch.arange(300, device="cuda")).to(torch.int32)
    b = problem(torch, [4, 4], [700, 90], [33] * 8, 8, 2, 128, 16, torch.bfloat16)
    c = problem(torch, [9], None, [1000] * 9, 8, 2, 64, 32, torch.float16)
    ws = torch.full((q4.q4_prefix_attn_workspace(300, 2, 8, 2, 128),), 255, device="cuda", dtype=torch.uint8)
    for p in (a, b, c, a, c, b):
        check(torch, p, ws=ws, flags=q4.Q4_RUN_OVERLAPPED)


@pytest.mark.parametrize("D", [64, 128])
def test_a_large_batch_is_the_same_every_time(torch, D):
    """Every SM with several segments of both kinds, over and over with no wait between the calls:
    what a register, a stage or a part holds too early or too late shows as another result."""
    S = 192
    own = [(37 * i) % 300 for i in range(S)]
    p = problem(torch, [S], [5000], own, 32, 8, D, 64, torch.bfloat16, stale=False)
    ws = torch.empty(q4.q4_prefix_attn_workspace(S, 1, 32, 8, D), device="cuda", dtype=torch.uint8)
    first, lse = run(torch, p, ws=ws)
    again = [run(torch, p, ws=ws) for _ in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, a) and torch.equal(lse, b) for a, b in again)
    check(torch, {n: (v[:8] if n in ("q", "own_pages", "own_lens") else v) for n, v in p.items()} |
          {"group_offsets": torch.tensor([0, 8], device="cuda", dtype=torch.int32)})
