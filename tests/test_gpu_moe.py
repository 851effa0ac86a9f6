"""GPU parity of the mixture-of-experts operators against plain 64-bit forms
(moe_reference.py, which also derives the error bounds).
"""
import moe_reference as ref
import numpy as np
import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def to(torch, a, dtype=None):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.cuda() if dtype is None else t.to(dtype).cuda()


def work(torch, n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def num(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound, what):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    bad = ~(same | (np.abs(got - want) <= bound))
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, bound {np.broadcast_to(bound, got.shape)[i]!r}")


# ---------------------------------------------------------------- route

def run_route(torch, logits, k, score, renorm, scale=1.0, bias=None, mask=None):
    T, E = logits.shape
    i = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, off, rows, pos = i(T, k), i(E + 1), i(T * k), i(T, k)
    w = torch.full((T, k), 77.0, device="cuda")
    q4.q4moe_route_run(to(torch, logits), ids, w, off, rows, pos, work(torch, q4.q4moe_route_workspace(T, E, k)),
                       bias=to(torch, bias), token_mask=to(torch, mask), renormalize=renorm, scale=scale,
                       score=q4.Q4_ROUTE_SIGMOID if score == "sigmoid" else q4.Q4_ROUTE_SOFTMAX)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (ids, w, off, rows, pos)]


def check_route(torch, logits, k, score, renorm, **kw):
    ids, w, off, rows, pos = run_route(torch, logits, k, score, renorm, **kw)
    e_ids, e_w, e_off, e_rows, e_pos, rel = ref.route(logits, k, score, renorm, **kw)
    for name, got, want in (("ids", ids, e_ids), ("offsets", off, e_off), ("rows", rows, e_rows), ("pos", pos, e_pos)):
        assert np.array_equal(got, want), name
    within(w.astype(np.float64), e_w, rel * np.abs(e_w) + 1e-37, "weights")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 4, 4), (17, 33, 5), (128, 64, 8), (129, 64, 8),
                                   (40, 256, 7), (300, 257, 9), (65, 1000, 32), (1031, 128, 8), (2100, 24, 1)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route(torch, T, E, k, score, renorm):
    rng = np.random.default_rng(T * 1009 + E)
    logits = rng.normal(0, 2, (T, E)).astype(np.float32)
    check_route(torch, logits, k, score, renorm, scale=2.5)
    bias = rng.normal(0, 1, E).astype(np.float32)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    logits[mask == 0] = NAN
    check_route(torch, logits, k, score, renorm, bias=bias, mask=mask)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_route_ties_and_masked_logits(torch, score, renorm):
    low = np.finfo(np.float32).min
    logits = np.array([[0.0] * 8, [-0.0, 0.0, -0.0, 0.0, 1.0, 1.0, -1.0, -1.0], [-INF] * 8, [NAN] * 8,
                       [-INF, 2.0, -INF, 2.0, NAN, -INF, -INF, -INF], [low] * 8,
                       [low, low, 5.0, low, -INF, low, NAN, low], [80.0, -80.0, 0.0, 1e30, -1e30, 3.0, 2.0, 1.0],
                       [0.0, 1e-45, -1e-45, 0.0, 0.0, 0.0, 0.0, 0.0]], np.float32)
    with np.errstate(over="ignore"):
        check_route(torch, logits, 3, score, renorm)
        check_route(torch, logits, 8, score, renorm)
    # a bias that hides an expert, and one that makes it the first choice of everybody
    bias = np.array([0, 0, 0, -INF, 0, 0, 100, 0], np.float32)
    check_route(torch, np.random.default_rng(3).normal(0, 1, (50, 8)).astype(np.float32), 3, score, renorm, bias=bias)


def test_route_all_tokens_masked(torch):
    logits = np.zeros((200, 16), np.float32)
    check_route(torch, logits, 6, "softmax", True, mask=np.zeros(200, np.uint8))
    check_route(torch, logits[:5], 6, "softmax", True, mask=np.zeros(5, np.uint8))


# ---------------------------------------------------------------- experts

def make_weights(rng, E, N, K, g, sym):
    nb = K // g
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales = rng.uniform(0.005, 0.02, (E, N, nb)).astype(np.float16)
    zeros = None
    if not sym:
        zeros = rng.integers(0, 256, (E, N, (nb + 1) // 2), dtype=np.uint8)
    return codes, scales, zeros


def groups(rng, E, k, T, shape):
    """offsets and rows of T tokens with k choices: even, skewed to one expert, or with empty experts."""
    if shape == "one":
        ids = np.full((T, k), E // 2)
    elif shape == "holes":
        ids = rng.integers(0, max(1, E // 2), (T, k)) * 2 % E
    else:
        ids = rng.integers(0, E, (T, k))
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.array([(flat < e).sum() for e in range(E + 1)], np.int32)
    return offsets, (order // k).astype(np.int32)


def run_experts(torch, weights, g, x, rows, offsets, R, swiglu, bf16, fill=7.0, stream=None, shift=0, **kw):
    codes, scales, zeros = weights
    E, N, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    t = torch.bfloat16 if bf16 else torch.float32
    ct, st = to(torch, codes), to(torch, scales)
    if shift:   # scales at an address that is a multiple of 2 only
        buf = torch.empty(st.numel() + shift, dtype=torch.float16, device="cuda")
        buf[shift:] = st.reshape(-1)
        st = buf[shift:].reshape(st.shape)
    zt = to(torch, zeros)
    xt, rt, ot = to(torch, x, t), to(torch, rows), to(torch, offsets)
    y = torch.full((R, N // 2 if swiglu else N), fill, dtype=t, device="cuda")
    ws = work(torch, q4.q4moe_gemm_workspace(R, x.shape[0], N, K, E, t))
    q4.q4moe_gemm_run(ct, st, zt, xt, rt, ot, y, ws, group=g, stream=stream,
                      epilogue=q4.Q4_EPILOGUE_SWIGLU if swiglu else q4.Q4_EPILOGUE_NONE, **kw)
    torch.cuda.synchronize()
    assert q4.q4gemv_device_status() == q4.Q4_OK
    return y


def check_experts(torch, seed, E, k, T, N, K, g, sym, swiglu, bf16, shape="even", gather=True, x=None, shift=0):
    rng = np.random.default_rng(seed)
    weights = make_weights(rng, E, N, K, g, sym)
    offsets, rows = groups(rng, E, k, T, shape)
    R = T * k
    if x is None:
        x = rng.normal(0, 1, (T if gather else R, K))
    x = num(torch.from_numpy(x).to(torch.bfloat16 if bf16 else torch.float32))
    rows = rows if gather else None
    y = run_experts(torch, weights, g, x, rows, offsets, R, swiglu, bf16, shift=shift)
    want, bound = ref.experts(ref.dequant(*weights, g), x, rows, offsets, np.full(tuple(y.shape), 7.0), swiglu, bf16)
    within(num(y), want, bound, "y")


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,k,T,N,K,g", [
    (1, 1, 1, 1, 32, 32), (1, 1, 3, 7, 64, 64), (4, 2, 1, 130, 96, 32), (8, 2, 5, 128, 128, 128),
    (8, 4, 9, 300, 160, 32), (6, 3, 40, 257, 832, 64), (3, 1, 100, 129, 896, 128), (16, 2, 33, 64, 4864, 32),
    (2, 2, 150, 200, 1152, 128), (64, 8, 16, 96, 256, 32), (5, 1, 700, 260, 320, 64), (40, 1, 40, 512, 2048, 128)])
def test_experts_sizes(torch, bf16, E, k, T, N, K, g):
    for sym, gather in ((True, True), (False, False)):
        check_experts(torch, E + T, E, k, T, N, K, g, sym, False, bf16, gather=gather)
    if N % 2 == 0:
        check_experts(torch, E + T, E, k, T, N, K, g, False, True, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape,T", [("one", 1), ("one", 17), ("one", 300), ("holes", 64), ("holes", 260)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_experts_uneven(torch, bf16, shape, T, swiglu):
    check_experts(torch, T, 9, 2, T, 192, 512, 64, False, swiglu, bf16, shape=shape)


@pytest.mark.parametrize("T", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513])
def test_experts_rows_around_tile_edges(torch, T):
    check_experts(torch, T, 3, 1, T, 140, 256, 32, False, False, T % 2 == 0, shape="one")


def test_experts_scales_at_odd_addresses(torch):
    for K, g in ((896, 128), (2048, 128), (1024, 32)):
        check_experts(torch, K, 4, 2, 20, 136, K, g, False, False, False, shift=1)
        check_experts(torch, K, 4, 2, 20, 136, K, g, True, True, True, shift=3)


@pytest.mark.parametrize("bf16", [False, True])
def test_experts_range_of_activations(torch, bf16):
    """Rows far beyond binary16's range, tiny rows, zero rows, and rows of mixed sizes."""
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (24, 256))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0.0
    x[3] *= 70000.0
    x[4, ::2] *= 1e4
    x[5, 7] = 3e9
    x[6] *= 1e-41 if not bf16 else 1e-36   # binary32 subnormals
    x[7, 1:] = 0.0
    check_experts(torch, 5, 4, 1, 24, 132, 256, 32, False, False, bf16, x=x)


def test_experts_ignore_what_no_expert_reads(torch):
    """Unowned rows of y stay, NaN in unread rows of x stays out, bad offsets and row indexes stay inside."""
    rng = np.random.default_rng(11)
    weights = make_weights(rng, 5, 96, 128, 32, False)
    W = ref.dequant(*weights, 32)
    x = rng.normal(0, 1, (30, 128)).astype(np.float32)
    x[20:] = NAN
    rows = rng.integers(0, 20, 60).astype(np.int32)
    rows[50:] = 25                                   # rows that no expert owns point at NaN
    for offsets in ([0, 10, 10, 31, 40, 50], [3, 3, 20, 20, 44, 47], [0, 0, 0, 0, 0, 0], [-5, 4, 9, 9, 60, 700],
                    [0, 30, 20, 25, 25, 40]):
        offsets = np.array(offsets, np.int32)
        r = rows.copy()
        r[5], r[33] = -1, 2 ** 31 - 1                # read as rows of zeros
        if offsets[-1] > 50:
            r[50:] = 3
        got = num(run_experts(torch, weights, 32, x, r, offsets, 60, False, False))
        want, bound = ref.experts(W, x, r, offsets, np.full(got.shape, 7.0), False, False)
        within(got, want, bound, f"offsets {offsets.tolist()}")


def test_experts_non_finite_rows_stay_alone(torch):
    """A row of x with NaN or infinity spoils its own outputs and no other row's."""
    rng = np.random.default_rng(12)
    weights = make_weights(rng, 2, 64, 64, 32, True)
    x = rng.normal(0, 1, (9, 64)).astype(np.float32)
    x[4, 3], x[6, 9] = NAN, INF
    offsets = np.array([0, 5, 9], np.int32)
    got = num(run_experts(torch, weights, 32, x, None, offsets, 9, False, False))
    clean = np.where(np.isfinite(x), x, 0.0)
    want, bound = ref.experts(ref.dequant(*weights, 32), clean, None, offsets, np.zeros(got.shape), False, False)
    ok = np.isfinite(x).all(axis=1)
    within(got[ok], want[ok], bound[ok], "finite rows")
    assert not np.isfinite(got[4]).any()
    assert not np.isfinite(got[6]).any()


def test_experts_past_32_bits(torch):
    """The last expert's codes lie beyond 4 GB."""
    E, N, K, g = 21, 28672, 14336, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    assert (E - 1) * N * K // 2 > 2 ** 32 - 2 ** 28
    scales = torch.full((E, N, K // g), 0.01, dtype=torch.float16, device="cuda")
    scales[-1] = (torch.rand(N, K // g, device="cuda", generator=gen) * 0.02).half()
    x = torch.randn(3, K, device="cuda", generator=gen)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 3
    y = torch.empty(3, N, device="cuda")
    q4.q4moe_gemm_run(codes, scales, None, x, None, offsets, y, work(torch, q4.q4moe_gemm_workspace(3, 3, N, K, E, x.dtype)),
                      group=g)
    torch.cuda.synchronize()
    part = slice(N - 300, N)
    W = ref.dequant(codes[-1:, part].cpu().numpy(), scales[-1:, part].cpu().numpy(), None, g)
    want, bound = ref.experts(W, num(x), None, np.array([0, 3]), np.zeros((3, 300)), False, False)
    within(num(y[:, part]), want, bound, "last rows of the last expert")


def test_experts_repeat_exactly(torch):
    """The same call twice, and with another workspace content: bit for bit."""
    rng = np.random.default_rng(21)
    weights = make_weights(rng, 8, 320, 1024, 32, False)
    offsets, rows = groups(rng, 8, 2, 50, "even")
    x = rng.normal(0, 1, (50, 1024))
    a = run_experts(torch, weights, 32, x, rows, offsets, 100, False, False)
    for _ in range(3):
        torch.full((1 << 24,), NAN, device="cuda")   # (what an allocator hands out next)
        assert torch.equal(a, run_experts(torch, weights, 32, x, rows, offsets, 100, False, False))


def test_experts_in_a_graph_and_on_a_stream(torch):
    """Captured once, replayed for other groups and activations; inputs made on the same side stream."""
    rng = np.random.default_rng(31)
    E, N, K, g, R = 6, 200, 512, 64, 48
    weights = make_weights(rng, E, N, K, g, False)
    codes, scales, zeros = (to(torch, a) for a in weights)
    W = ref.dequant(*weights, g)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.zeros(24, K, device="cuda")
        rows = torch.zeros(R, dtype=torch.int32, device="cuda")
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        y = torch.zeros(R, N, device="cuda")
        ws = work(torch, q4.q4moe_gemm_workspace(R, 24, N, K, E, x.dtype))
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            q4.q4moe_gemm_run(codes, scales, zeros, x, rows, offsets, y, ws, group=g)
        for shape in ("even", "one", "holes"):
            o, r = groups(rng, E, 2, 24, shape)
            xn = rng.normal(0, 1, (24, K)).astype(np.float32)
            x.copy_(to(torch, xn))
            rows.copy_(to(torch, r))
            offsets.copy_(to(torch, o))
            graph.replay()
            s.synchronize()
            want, bound = ref.experts(W, xn, r, o, np.zeros((R, N)), False, False)
            within(num(y), want, bound, shape)


# ---------------------------------------------------------------- block norm

def check_norm(torch, seed, T, H, k, bf16, post, gate, pre, drop=0.2, alpha=0.7, eps=1e-6, y=None, odd_gate=False):
    rng = np.random.default_rng(seed)
    t = torch.bfloat16 if bf16 else torch.float32
    cast = lambda a: num(torch.from_numpy(np.asarray(a)).to(t))  # noqa: E731
    R = T * k if k else T
    y = cast(rng.normal(0, 1, (R, H)) if y is None else y)
    x = cast(rng.normal(0, 2, (T, H)))
    pos = weights = None
    if k:
        pos = rng.permutation(R).reshape(T, k).astype(np.int32)
        pos[rng.random((T, k)) < drop] = -1
        weights = rng.random((T, k)).astype(np.float32)
    post = rng.uniform(0.5, 1.5, H).astype(np.float32) if post else None
    pre = rng.uniform(0.5, 1.5, H).astype(np.float32) if pre else None
    gate = None if gate is None else cast(rng.normal(1, 0.3, (T, H) if gate == "token" else (H,)))
    gt = to(torch, gate, t)
    if odd_gate:
        buf = torch.empty(gt.numel() + 1, dtype=t, device="cuda")
        buf[1:] = gt.reshape(-1)
        gt = buf[1:].reshape(gt.shape)
    out = torch.full((T, H), 9.0, dtype=t, device="cuda")
    a = torch.full((T, H), 9.0, dtype=t, device="cuda") if pre is not None else None
    q4.q4_block_norm_run(to(torch, y, t), to(torch, x, t), out, pos=to(torch, pos), weights=to(torch, weights),
                         post_gamma=to(torch, post), gate=gt, residual_scale=alpha, pre_gamma=to(torch, pre),
                         out_norm=a, eps=eps)
    torch.cuda.synchronize()
    half = ref.UBF if bf16 else ref.U32
    want, b1, wa, b2 = ref.block_norm(y, x, pos, weights, post, gate, np.float32(alpha).astype(np.float64), pre,
                                      float(np.float32(eps)), half)
    within(num(out), want, b1, "out")
    if a is not None:
        within(num(a), wa, b2, "out_norm")


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,H,k", [(1, 1, 1), (2, 7, 2), (1, 4096, 8), (5, 896, 0), (9, 1000, 3), (33, 2047, 4),
                                   (4, 8192, 2), (3, 16384, 1), (2, 16383, 2), (700, 64, 32)])
def test_norm_sizes(torch, bf16, T, H, k):
    for post, gate, pre in ((True, "token", True), (False, None, False), (True, "channel", False),
                            (False, "channel", True)):
        check_norm(torch, T + H, T, H, k, bf16, post, gate, pre)


@pytest.mark.parametrize("bf16", [False, True])
def test_norm_token_without_rows(torch, bf16):
    check_norm(torch, 3, 6, 512, 4, bf16, True, "token", True, drop=1.0)
    check_norm(torch, 4, 6, 512, 4, bf16, False, None, True, drop=1.0)


def test_norm_skips_what_pos_leaves_out(torch):
    """NaN and infinity in rows that no pos names, and pos beyond the rows."""
    y = torch.randn(8, 256, device="cuda")
    y[5], y[6] = NAN, INF
    x = torch.randn(3, 256, device="cuda")
    pos = torch.tensor([[0, 1], [-1, 8], [2 ** 31 - 1, 4]], dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    out = torch.empty_like(x)
    q4.q4_block_norm_run(y, x, out, pos=pos, weights=w)
    want = torch.stack([x[0].double() + y[0].double() + y[1].double(), x[1].double(), x[2].double() + y[4].double()])
    assert float((out.double() - want).abs().max()) <= 3 * 2.0 ** -24 * 16


def test_norm_unaligned_gate(torch):
    for bf16 in (False, True):
        check_norm(torch, 8, 5, 640, 2, bf16, True, "channel", True, odd_gate=True)
        check_norm(torch, 9, 5, 640, 2, bf16, True, "token", True, odd_gate=True)


# ---------------------------------------------------------------- the block

@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k,H,inner,g", [(1, 8, 2, 256, 128, 32), (7, 16, 4, 384, 64, 64), (150, 12, 3, 256, 256, 128)])
def test_block_equals_its_parts(torch, bf16, T, E, k, H, inner, g):
    """q4moe_block_run gives bit for bit what the four calls give one after another."""
    rng = np.random.default_rng(T)
    t = torch.bfloat16 if bf16 else torch.float32
    up = [to(torch, a) for a in make_weights(rng, E, 2 * inner, H, g, False)]
    down = [to(torch, a) for a in make_weights(rng, E, H, inner, g, True)]
    logits = to(torch, rng.normal(0, 1, (T, E)).astype(np.float32))
    a, x = to(torch, rng.normal(0, 1, (T, H)), t), to(torch, rng.normal(0, 1, (T, H)), t)
    post, pre = (to(torch, rng.uniform(0.5, 1.5, H).astype(np.float32)) for _ in range(2))
    gate = to(torch, rng.normal(1, 0.2, (T, H)), t)
    mask = to(torch, (rng.random(T) < 0.8).astype(np.uint8))
    i32 = dict(dtype=torch.int32, device="cuda")

    def outs():
        return torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    ids, w, out, nrm = outs()
    flags = q4.Q4_RUN_OVERLAPPED if T > 1 else None
    q4.q4moe_block_run(up, down, logits, a, x, out, nrm, ids, w,
                       work(torch, q4.q4moe_block_workspace(T, E, k, H, inner, t)), group=g, token_mask=mask,
                       post_gamma=post, gate=gate, residual_scale=0.5, pre_gamma=pre, route_scale=1.5, flags=flags)
    ids2, w2, out2, nrm2 = outs()
    off, rows, pos = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T, k, **i32)
    h, y = torch.zeros(T * k, inner, dtype=t, device="cuda"), torch.zeros(T * k, H, dtype=t, device="cuda")
    q4.q4moe_route_run(logits, ids2, w2, off, rows, pos, work(torch, q4.q4moe_route_workspace(T, E, k)),
                       token_mask=mask, scale=1.5)
    q4.q4moe_gemm_run(*up, a, rows, off, h, work(torch, q4.q4moe_gemm_workspace(T * k, T, 2 * inner, H, E, t)), group=g,
                      epilogue=q4.Q4_EPILOGUE_SWIGLU)
    q4.q4moe_gemm_run(*down, h, None, off, y, work(torch, q4.q4moe_gemm_workspace(T * k, T * k, H, inner, E, t)), group=g)
    q4.q4_block_norm_run(y, x, out2, pos=pos, weights=w2, post_gamma=post, gate=gate, residual_scale=0.5,
                         pre_gamma=pre, out_norm=nrm2)
    torch.cuda.synchronize()
    for p, q in ((ids, ids2), (w, w2), (out, out2), (nrm, nrm2)):
        assert torch.equal(p, q)
    assert torch.isfinite(out).all() and torch.isfinite(nrm).all()


# ---------------------------------------------------------------- bounded waits, checked indexes

@pytest.mark.parametrize("bf16,T", [(False, 9), (False, 200), (True, 9), (True, 200)])
def test_experts_bounded_wait_reports_timeout_without_fault(torch, bf16, T):
    """A zero bound makes the pipelines give up; the context and the next call are sound."""
    rng = np.random.default_rng(T)
    weights = make_weights(rng, 4, 300, 1024, 64, False)
    offsets, rows = groups(rng, 4, 2, T, "even")
    x = num(torch.from_numpy(rng.normal(0, 1, (T, 1024))).to(torch.bfloat16 if bf16 else torch.float32))
    t = torch.bfloat16 if bf16 else torch.float32
    args = [to(torch, a) for a in weights] + [to(torch, x, t), to(torch, rows), to(torch, offsets)]
    y = torch.zeros(2 * T, 300, dtype=t, device="cuda")
    ws = work(torch, q4.q4moe_gemm_workspace(2 * T, T, 300, 1024, 4, t))
    q4.q4moe_gemm_run(*args, y, ws, group=64, wait_timeout_ns=0)
    torch.cuda.synchronize()
    assert q4.q4gemv_device_status() == q4.Q4_ERR_TIMEOUT
    assert q4.q4gemv_device_status() == q4.Q4_OK        # reported once
    q4.q4moe_gemm_run(*args, y, ws, group=64)
    torch.cuda.synchronize()
    want, bound = ref.experts(ref.dequant(*weights, 64), x, rows, offsets, np.zeros((2 * T, 300)), False, bf16)
    within(num(y), want, bound, "after the timeout")


@pytest.fixture(scope="module")
def checking(torch):
    """The bounds-checking build in the library's place."""
    from gemm_decode_gb300 import build as q4build
    path = q4build.build(variant="check")
    saved = q4._lib, q4.library_path
    q4._lib, q4.library_path = None, lambda: path
    try:
        assert q4.q4gemv_bounds_violations() == 0
        yield
    finally:
        q4._lib, q4.library_path = saved


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,k,T,N,K,g", [(9, 2, 70, 330, 416, 32), (4, 2, 5, 257, 2112, 64), (2, 1, 300, 514, 896, 128)])
def test_experts_stay_in_bounds(torch, checking, bf16, E, k, T, N, K, g):
    check_experts(torch, E, E, k, T, N, K, g, False, False, bf16, shape="holes")
    assert q4.q4gemv_bounds_violations() == 0


# ---------------------------------------------------------------- the example

@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_example_block(torch, dtype):
    """The example's block against a plain one, for a prompt and for single tokens in a graph."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block
    worst = moe_block.check(getattr(torch, dtype), hidden=512, inner=256, experts=8, top_k=2, group=64)
    # bfloat16: the rows inside an expert and its output are rounded too (2^-8 half steps each)
    assert worst <= (4 * ref.UBF if dtype == "bfloat16" else 1e-5)
