"""The router beyond test_gpu_moe.py: a bias on the score, against a plain form in 64 bits."""
import numpy as np
import pytest
from gpu_util import torch_cuda
from test_gpu_moe import to, within, work

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
KIND = {"softmax": q4.Q4_ROUTE_SOFTMAX, "sigmoid": q4.Q4_ROUTE_SIGMOID}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def run(torch, logits, k, score, renorm, bias=None, mask=None, scale=1.0):
    T, E = logits.shape
    i = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, off, rows, pos = i(T, k), i(E + 1), i(T * k), i(T, k)
    w = torch.full((T, k), 77.0, device="cuda")
    q4.q4moe_route_run(to(torch, logits), ids, w, off, rows, pos, work(torch, q4.q4moe_route_workspace(T, E, k)),
                       bias=to(torch, bias), token_mask=to(torch, mask), renormalize=renorm, scale=scale, score=score)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (ids, w, off, rows, pos)]


def scores(logits, kind):
    l = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    if kind == "sigmoid":
        return 1.0 / (1.0 + np.exp(-l))
    high = l.max(axis=1, keepdims=True)
    p = np.exp(l - np.where(np.isfinite(high), high, 0.0))
    return p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)


def grouped(ids, E):
    """offsets, rows and pos of chosen ids: the choices stably sorted by expert."""
    T, k = ids.shape
    flat = np.where(ids < 0, E, ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[order], np.arange(E + 1)).astype(np.int32)
    rows = np.where(np.arange(T * k) < offsets[E], order // k, -1).astype(np.int32)
    pos = np.empty(T * k, np.int32)
    pos[order] = np.arange(T * k)
    return offsets, rows, np.where(ids < 0, -1, pos.reshape(T, k)).astype(np.int32)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_bias_on_the_score_by_hand(torch, kind):
    """Rows where score + bias and logit + bias choose differently, ties, and experts that no bias brings back."""
    logits = np.array([[4.0, 0.0, -2.0, -9.0], [1.0, 1.0, 1.0, 1.0], [-INF, NAN, 0.5, -INF], [9.0, 9.0, -9.0, 9.0]],
                      np.float32)
    bias = np.array([0.0, 0.99, 0.0, 1.5], np.float32)
    s = KIND[kind] | q4.Q4_ROUTE_SCORE_BIAS
    ids, w, off, rows, pos = run(torch, logits, 2, s, False, bias)
    # (softmax scores of the first row: 0.979, 0.018, ...; sigmoids 0.982, 0.5, ...)
    assert ids.tolist() == [[3, 1], [3, 1], [2, -1], [3, 1]]
    p = scores(logits, kind)
    want = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0.0)
    within(w.astype(np.float64), want, 40 * U32 * want + 1e-37, "weights")
    for got, e in zip((off, rows, pos), grouped(ids, 4)):
        assert np.array_equal(got, e)
    # logit + bias: the first row's 4.0 stays ahead of everything
    assert run(torch, logits, 2, KIND[kind], False, bias)[0][0].tolist() == [0, 1]
    # equal scores and biases: the lower expert
    assert run(torch, np.zeros((1, 40), np.float32), 4, s, True, np.ones(40, np.float32))[0].tolist() == [[0, 1, 2, 3]]
    # a bias of -inf or NaN hides an expert, no bias at all: the score's own order
    hide = np.array([-INF, 0.0, NAN, 0.0], np.float32)
    assert run(torch, logits[:1], 3, s, True, hide)[0].tolist() == [[1, 3, -1]]
    assert run(torch, logits[:1], 3, s, True)[0].tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 33, 4), (129, 256, 8), (2000, 128, 8), (40, 1000, 32)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_bias_on_the_score(torch, T, E, k, kind, renorm):
    rng = np.random.default_rng(T + E)
    logits = rng.normal(0, 2, (T, E)).astype(np.float32)
    bias = rng.normal(0, 0.2, E).astype(np.float32)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[0] = 1
    logits[mask == 0] = NAN
    logits[:, E // 2] = -INF
    ids, w, off, rows, pos = run(torch, logits, k, KIND[kind] | q4.Q4_ROUTE_SCORE_BIAS, renorm, bias, mask, scale=2.5)
    live = mask != 0
    assert (ids[~live] == -1).all() and (w[~live] == 0).all() and (pos[~live] == -1).all()
    p = scores(logits, kind)
    ok = np.isfinite(logits)
    spread = np.where(ok, logits, -np.inf).max(axis=1, initial=0.0) - np.where(ok, logits, np.inf).min(axis=1, initial=0.0)
    # a score is off by a few steps of binary32 (expf 2 ulp, E additions, a division), and is
    # rounded once more with the bias added; two sums nearer than that may change places
    off_by = (E + 20 + 2 * spread) * U32 * p.max(axis=1) + 2 * U32 * (1.0 + np.abs(bias).max())
    sel = np.where(np.isneginf(logits) | np.isnan(logits), -np.inf, p + bias.astype(np.float64))
    for t in np.nonzero(live)[0]:
        chosen = ids[t]
        assert len(set(chosen.tolist())) == k and (chosen >= 0).all()
        got = sel[t, chosen]
        assert (np.diff(got) <= 2 * off_by[t]).all(), "descending"
        assert np.delete(sel[t], chosen).max() <= got.min() + 2 * off_by[t], "the largest"
    v = np.take_along_axis(p, np.maximum(ids, 0), 1)
    if renorm:
        v = v / (v.sum(axis=1, keepdims=True) + (1e-20 if kind == "sigmoid" else 1e-300))
    within(w[live].astype(np.float64), 2.5 * v[live], (E + 60) * U32 * 2.5 * v[live] + 1e-37, "weights")
    for got, e in zip((off, rows, pos), grouped(ids, E)):
        assert np.array_equal(got, e)


def long_prompt(torch, T, E, k, seed):
    """Logits, mask, and the chosen experts by a plain stable sort."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(T, E, device="cuda", generator=g)
    logits[:, E // 3] += 2.0
    mask = (torch.rand(T, device="cuda", generator=g) < 0.9).to(torch.uint8)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    ids[mask == 0] = -1
    return logits, mask, ids


# blocks of 512 // k tokens: 256 and 257 of them, several thousand, a last one that is not full
@pytest.mark.parametrize("T,E,k", [(4096, 40, 32), (4097, 40, 32), (80003, 40, 32), (300000, 8, 8), (131071, 1000, 16),
                                   (270000, 3, 2)])
def test_order_of_long_prompts(torch, T, E, k):
    logits, mask, ids = long_prompt(torch, T, E, k, T)
    i = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    got, off, rows, pos = i(T, k), i(E + 1), i(T * k), i(T, k)
    w = torch.empty(T, k, device="cuda")
    n = q4.q4moe_route_workspace(T, E, k)
    ws = work(torch, n + 4096)
    ws[n:] = 77
    q4.q4moe_route_run(logits, got, w, off, rows, pos, ws[:n], token_mask=mask)
    assert torch.equal(got, ids)
    for have, want in zip((off, rows, pos), grouped(ids.cpu().numpy(), E)):
        assert np.array_equal(have.cpu().numpy(), want)
    assert bool((ws[n:] == 77).all())


def test_time_grows_with_the_tokens(torch):
    """Four times the tokens take no more than about four times as long (each block's own sum
    over all blocks would take sixteen times as long)."""
    def best(T, E=128, k=8):
        logits, mask, ids = long_prompt(torch, T, E, k, 1)
        outs = [torch.empty_like(ids), torch.empty(T, k, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty_like(ids),
                work(torch, q4.q4moe_route_workspace(T, E, k))]
        times = []
        for _ in range(8):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            q4.q4moe_route_run(logits, *outs, token_mask=mask)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        return min(times[2:])
    few, many = best(1 << 18), best(1 << 20)
    assert many <= 8 * few, (few, many)


@pytest.mark.parametrize("flag", [0, q4.Q4_ROUTE_SCORE_BIAS])
def test_sigmoids_of_far_logits(torch, flag):
    """Renormalised sigmoids of logits where exp(-l) overflows: s / (sum s + 1e-20)."""
    logits = np.array([[-90.0, -91.0, -95.0, -99.0], [-88.0, -100.0, -3.0e4, -95.0], [90.0, -90.0, 200.0, -89.0]], np.float32)
    ids, w, *_ = run(torch, logits, 3, q4.Q4_ROUTE_SIGMOID | flag, True, bias=np.zeros(4, np.float32) if flag else None)
    assert ids[:2].tolist() == [[0, 1, 2], [0, 3, 1]] and (ids[2] != 3).sum() >= 2
    s = 1.0 / (1.0 + np.exp(-np.take_along_axis(logits, ids, 1).astype(np.float64)))
    want = s / (s.sum(axis=1, keepdims=True) + 1e-20)
    # binary32's last step, 2^-149, where s is subnormal
    within(w.astype(np.float64), want, want * (60 * U32 + 2.0 ** -149 / np.maximum(s, 2.0 ** -149)) + 1e-37, "weights")
    alone = run(torch, logits[:, :1], 1, q4.Q4_ROUTE_SIGMOID | flag, False)[1]
    within(alone.astype(np.float64), 1.0 / (1.0 + np.exp(-logits[:, :1].astype(np.float64))), 60 * U32 + 0 * alone, "alone")
