"""Rotary positions and the cache's new rows against the formula in 64 bits."""
import decode_reference as ref
import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def pools(torch, pages, heads, page, D, t16, layout):
    """Two pools with every element a value of its own kind of garbage, in one of three layouts."""
    fill = lambda *n: torch.randn(*n, device="cuda").to(t16)  # noqa: E731
    if layout == "heads":      # [pages][heads][page][D]
        return fill(pages, heads, page, D), fill(pages, heads, page, D)
    if layout == "tokens":     # [pages][page][heads][D]
        return tuple(fill(pages, page, heads, D).transpose(1, 2) for _ in range(2))
    both = fill(pages, 2, heads, page, D)   # keys and values of a page side by side
    return both[:, 0], both[:, 1]


def check(torch, T, Hq, Hkv, D, rot, half, dtype, t16, norm=True, page=16, layout="heads", start=0, drop=0.0,
          scale=1.0, slots=True, odd=0, lead=0, keys=True, inv_freq=None, eps=1e-6):
    torch.manual_seed(T * 131 + D + rot)
    n = (Hq + 2 * Hkv) * D
    # rows of one product, `odd` more elements a row than the heads need, `lead` before the first
    flat = (2 * torch.randn(T * (n + odd) + lead, device="cuda")).to(dtype)
    qkv = flat[lead:].view(T, n + odd)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = qkv[:, (Hq + Hkv) * D:n].unflatten(1, (Hkv, D))
    positions = (start + torch.arange(T, device="cuda", dtype=torch.int64)).to(torch.int32)
    if inv_freq is None:
        inv_freq = q4.q4_rope_frequencies(rot, 10000.0)
    inv_freq = inv_freq.cuda()
    qg, kg = (0.5 + torch.rand(D, device="cuda") for _ in range(2)) if norm else (None, None)
    pages = (T + page - 1) // page + 2
    kc, vc = pools(torch, pages, Hkv, page, D, t16, layout)
    before = kc.clone(), vc.clone()
    where = None
    if slots:
        where = torch.randperm(pages * page, device="cuda")[:T].to(torch.int32)
        where[torch.rand(T, device="cuda") < drop] = -1
        if drop:
            where[0] = pages * page   # behind the pool: not written either
    q_out = torch.full((T, Hq, D), 7.0, device="cuda", dtype=t16)
    q4.q4_rope_append_run(q, k if keys else None, v if keys else None, positions, inv_freq, q_out,
                          kc if keys else None, vc if keys else None, slots=where if keys else None, q_gamma=qg,
                          k_gamma=kg if keys else None, layout=q4.Q4_ROPE_HALF if half else q4.Q4_ROPE_INTERLEAVED,
                          scale=scale, eps=eps)
    torch.cuda.synchronize()
    want, bound = ref.rope(q, qg, positions, inv_freq, half, scale, eps)
    ref.within(q_out, want, (1 + 2.0 ** -7) * bound + ref.rounding(want, t16), "q_out")
    if not keys:
        return q_out
    want, bound = ref.rope(k, kg, positions, inv_freq, half, scale, eps)
    at = where.long().cpu() if slots else torch.arange(T)
    live = (at >= 0) & (at < pages * page)
    rows = lambda c: c.transpose(1, 2).reshape(pages * page, Hkv, D).cpu()  # noqa: E731
    ref.within(rows(kc)[at[live]], want[live], ((1 + 2.0 ** -7) * bound + ref.rounding(want, t16))[live], "keys")
    assert torch.equal(rows(vc)[at[live]], v.float().to(t16).cpu()[live])
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[at[live]] = False
    for c, b in zip((kc, vc), before):
        assert torch.equal(rows(c)[rest], rows(b)[rest])   # every other row of the pools as it was
    return q_out


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("t16", ["bfloat16", "float16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,half", [
    (1, 1, 1, 64, 64, True), (1, 32, 8, 128, 128, True), (4, 32, 8, 128, 128, False), (33, 14, 2, 64, 32, False),
    (7, 28, 4, 128, 64, True), (5, 3, 3, 80, 80, True), (5, 6, 2, 96, 48, True), (3, 8, 1, 256, 64, False),
    (3, 2, 1, 256, 256, True), (9, 5, 5, 64, 24, True), (2, 4, 4, 64, 0, True), (2, 3, 1, 17, 16, False),
    (2, 3, 1, 6, 2, True), (1, 1, 1, 1, 0, True), (130, 64, 1, 64, 16, False), (2, 71, 13, 128, 128, True)])
def test_rope_against_the_formula(torch, T, Hq, Hkv, D, rot, half, dtype, t16):
    dtype, t16 = getattr(torch, dtype), getattr(torch, t16)
    check(torch, T, Hq, Hkv, D, rot, half, dtype, t16, norm=True, drop=0.3, layout="tokens")
    check(torch, T, Hq, Hkv, D, rot, half, dtype, t16, norm=False, slots=False, page=3, scale=1.25)


@pytest.mark.parametrize("layout", ["heads", "tokens", "paired"])
@pytest.mark.parametrize("odd,lead", [(0, 0), (8, 8), (1, 0), (0, 1), (4, 4)])
def test_rope_strides_and_alignments(torch, layout, odd, lead):
    for dtype in (torch.float32, torch.bfloat16):
        check(torch, 19, 8, 2, 128, 128, True, dtype, torch.bfloat16, layout=layout, odd=odd, lead=lead, page=5)


def test_rope_far_positions_keep_their_accuracy(torch):
    """Positions up to 2^31 - 1 and below zero: the angle is reduced exactly, so the bound of near
    ones holds.  (The reference's own reduction is good to 2^-22 turns there, so frequencies are
    multiples of 2^-20 turns' worth: exact in binary64 products.)"""
    for start in (131072 - 5, 10 ** 6, 2 ** 24 - 3, -17):
        check(torch, 9, 4, 2, 64, 64, True, torch.float32, torch.float16, start=start)
    f = torch.tensor([1.0, 0.5, 2.0 ** -10, 3e-5, 1e-30, 0.0, -0.25, 16.0])
    check(torch, 9, 4, 2, 64, 16, True, torch.float32, torch.float16, start=10 ** 7, inv_freq=f)


def test_rope_of_the_largest_position_by_integers(torch):
    """cos and sin at position 2^31 - 1 from a reduction in whole numbers on the host."""
    from fractions import Fraction
    from decimal import Decimal, getcontext
    import math
    getcontext().prec = 60
    two_pi = Fraction(Decimal("6.28318530717958647692528676655900576839433879875021164194989"))
    f = q4.q4_rope_frequencies(64, 500000.0)
    p = 2 ** 31 - 1
    x = torch.zeros(1, 1, 64, device="cuda")
    x[..., :32] = 1.0
    out = torch.empty(1, 1, 64, device="cuda", dtype=torch.float16)
    q4.q4_rope_append_run(x, None, None, torch.tensor([p], device="cuda", dtype=torch.int32), f.cuda(), out, None, None)
    for i in range(32):
        turns = Fraction(float(f[i])) * p / two_pi
        angle = float((turns - math.floor(turns)) * two_pi)
        for got, want in ((out[0, 0, i], math.cos(angle)), (out[0, 0, 32 + i], math.sin(angle))):
            assert abs(float(got) - want) <= 2.0 ** -21 + 2.0 ** -11 * abs(want) + 2.0 ** -25, i


def test_rope_queries_only_and_in_turns(torch):
    a = check(torch, 40, 32, 8, 128, 128, True, torch.bfloat16, torch.bfloat16, keys=False)
    b = check(torch, 40, 32, 8, 128, 128, True, torch.bfloat16, torch.bfloat16, keys=False)
    assert torch.equal(a, b)


def test_rope_of_rows_that_are_not_finite(torch):
    """A token with a NaN or an infinity spoils its own head alone, and values pass as they are."""
    T, H, D = 4, 2, 64
    x = torch.randn(T, 3 * H, D, device="cuda")
    x[1, 0, 5] = float("nan")
    x[2, H, 7] = float("inf")
    x[3, 2 * H, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")
    kc, vc = (torch.zeros(T, H, 1, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    out = torch.zeros(T, H, D, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(D, device="cuda")
    q4.q4_rope_append_run(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], torch.arange(T, device="cuda", dtype=torch.int32),
                          q4.q4_rope_frequencies(D).cuda(), out, kc, vc, q_gamma=g, k_gamma=g)
    fine = torch.isfinite(out).all(2)
    assert fine.cpu().tolist() == [[True, True], [False, True], [True, True], [True, True]]
    assert torch.isfinite(kc).all(3)[..., 0].cpu().tolist() == [[True, True], [True, True], [False, True], [True, True]]
    assert torch.equal(vc[:, :, 0].nan_to_num(9.0, 5.0, -5.0), x[:, 2 * H:].bfloat16().nan_to_num(9.0, 5.0, -5.0))


def test_rope_replayed_from_a_graph_with_other_positions(torch):
    T, Hq, Hkv, D = 3, 4, 2, 64
    qkv = torch.randn(T, Hq + 2 * Hkv, D, device="cuda")
    pos, slots = (torch.zeros(T, device="cuda", dtype=torch.int32) for _ in range(2))
    kc, vc = (torch.zeros(8, Hkv, 16, D, device="cuda", dtype=torch.float16) for _ in range(2))
    out = torch.zeros(T, Hq, D, device="cuda", dtype=torch.float16)
    f = q4.q4_rope_frequencies(D).cuda()
    call = lambda: q4.q4_rope_append_run(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, f, out, kc, vc,  # noqa: E731
                                         slots=slots, flags=q4.Q4_RUN_OVERLAPPED)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in (1, 50):
        qkv.normal_()
        pos.copy_(torch.arange(T) + step)
        slots.copy_(torch.tensor([step, 100 + step % 20, -1]))
        graph.replay()
        torch.cuda.synchronize()
        want, bound = ref.rope(qkv[:, :Hq], None, pos, f, True, 1.0, 1e-6)
        ref.within(out, want, bound * 1.01 + ref.rounding(want, torch.float16), "q_out")
        want, bound = ref.rope(qkv[:, Hq:Hq + Hkv], None, pos, f, True, 1.0, 1e-6)
        got = kc[step // 16, :, step % 16]
        ref.within(got, want[0], (bound * 1.01 + ref.rounding(want, torch.float16))[0], "keys")
