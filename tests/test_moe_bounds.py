"""The bounds of moe_bounds.py hold for a model of the kernels' arithmetic and tell it from
poorer ones: weights rounded to binary16, one part of x, x of 15 bits, one sum over all of K.
"""
import moe_bounds as mb
import numpy as np
import pytest


def make(K, group, N=192, rows=6, seed=0):
    rng = np.random.default_rng(seed + K)
    q, z = rng.integers(0, 16, (N, K)), np.repeat(rng.integers(0, 16, (N, K // group)), group, axis=1)
    s = rng.uniform(0.005, 0.02, (N, K // group)).astype(np.float16).astype(np.float64)
    return (q - z).astype(np.float64), s, rng.normal(0, 1, (rows, K)).astype(np.float32)


def cut(v):
    """Binary32 of v by cutting towards minus infinity, as an adder that drops the last bits."""
    m, e = np.frexp(v)
    return np.ldexp(np.floor(np.ldexp(m, 24)), e - 24)


def parts_of(x, bits=22):
    """The binary16 parts of each row scaled to [2^14, 2^15), and the scale back."""
    e = 14 - np.floor(np.log2(np.abs(x).max(axis=1, keepdims=True)))
    a = x.astype(np.float64) * 2.0 ** e
    if bits == 15:
        m, k = np.frexp(a)
        a = np.ldexp(np.round(np.ldexp(m, 15)), k - 15)
    hi = a.astype(np.float16).astype(np.float64)
    return [hi, (a - hi).astype(np.float16).astype(np.float64)][:1 if bits == 11 else 2], 2.0 ** -e


def model(d, s, x, group, weights16=False, bits=22, one_sum=False):
    """The kernel for few rows; or weights (q - z) s in binary16 and one sum over K."""
    parts, back = parts_of(x, bits)
    W = d
    if weights16 or one_sum:
        W = d * np.repeat(s, group, axis=1)
        if weights16:
            W = W.astype(np.float16).astype(np.float64)
        s = np.ones_like(s)
    K, total = d.shape[1], np.zeros((x.shape[0], d.shape[0]))
    for g0 in range(0, K, K if one_sum else group):
        n = K if one_sum else group
        acc = []
        for p in parts:
            v = np.zeros_like(total)
            for k in range(g0, g0 + n, 16):
                v = cut(v + p[:, k:k + 16] @ W[:, k:k + 16].T)
            acc.append(v)
        both = np.float32(sum(acc)).astype(np.float64)
        total = np.float32(total + s[:, g0 // group] * both).astype(np.float64)
    return total * back


def off(y, want):
    return np.linalg.norm(y - want) / np.linalg.norm(want)


@pytest.mark.parametrize("K,group", [(512, 64), (2048, 128), (2048, 32), (4864, 32), (4096, 128)])
def test_binary32_bounds_tell_the_kernel_from_poorer_ones(K, group):
    d, s, x = make(K, group)
    W = d * np.repeat(s, group, axis=1)
    want, b = mb.product(x.astype(np.float64), W, group, True, False)
    limit = mb.two_norm(K, group)
    right = model(d, s, x, group)
    assert off(right, want) <= limit and (np.abs(right - want) <= b).all()
    assert off(model(d, s, x, group, weights16=True), want) > 4 * limit
    assert off(model(d, s, x, group, bits=11), want) > 4 * limit
    assert off(model(d, s, x, group, bits=15), want) > 2 * limit
    if K >= 2048:   # (of a sum over 512 products little is cut)
        assert off(model(d, s, x, group, one_sum=True), want) > limit


def to_bf16(v):
    u = np.float32(v).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32).astype(np.float64)


def test_bfloat16_misroundings_tell_exact_weights_from_rounded_ones():
    K, group = 2048, 64
    d, s, x = make(K, group, N=600, rows=20)
    x = to_bf16(x).astype(np.float32)
    want = to_bf16(x.astype(np.float64) @ (d * np.repeat(s, group, axis=1)).T)
    share = lambda y: float((to_bf16(y) != want).mean())  # noqa: E731
    assert share(model(d, s, x, group, bits=11)) <= mb.MISROUNDED < share(model(d, s, x, group, bits=11, weights16=True)) / 4


def test_outliers_are_covered_by_the_absolute_term():
    """A row's largest element far above the others, under a zero weight: the others carry the
    error that the row's one scale leaves them, and no bound without the absolute term holds."""
    K, group = 512, 32
    d, s, x = make(K, group)
    d[:, 77] = 0.0
    x[:, 77] = 1e9
    W = d * np.repeat(s, group, axis=1)
    want, b = mb.product(x.astype(np.float64), W, group, True, False)
    got = model(d, s, x, group)
    assert (np.abs(got - want) <= b).all()
    assert off(got, want) > 2.0 ** -22 * 10
