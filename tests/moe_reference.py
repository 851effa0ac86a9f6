"""Plain 64-bit forms of the mixture-of-experts operators and the error each result may
carry, derived from the arithmetic the header states.

Half a step of a rounding, relative to the value: binary32 2^-24, binary16 2^-11, bfloat16
2^-8.  Tensor-core sums: binary32 accumulators, one addition per 16 products, which may cut
instead of round: 2^-23 each.
"""
import numpy as np

U32, U16, UBF = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


# ---------------------------------------------------------------- route

def route(logits, k, score, renorm, scale=1.0, bias=None, mask=None):
    """ids, weights (binary64), offsets, rows, pos and the relative error of the weights."""
    T, E = logits.shape
    sel = logits.astype(np.float32)
    if bias is not None:
        sel = (sel + bias.astype(np.float32)).astype(np.float32)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    rel = np.zeros((T, 1))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        ok = [e for e in range(E) if sel[t, e] > -np.inf]      # neither NaN nor -inf
        chosen = sorted(ok, key=lambda e: (-sel[t, e], e))[:k]
        if not chosen:
            continue
        l = logits[t].astype(np.float64)
        l[np.isnan(l)] = -np.inf
        if score == "softmax":
            pool = l[chosen] if renorm else l
            with np.errstate(invalid="ignore"):
                v = np.exp(l[chosen] - pool.max()) / np.exp(pool - pool.max()).sum()
            finite = l[chosen][np.isfinite(l[chosen])]
            spread = pool.max() - finite.min() if finite.size else 0.0
        else:
            with np.errstate(over="ignore"):
                v = 1.0 / (1.0 + np.exp(-l[chosen]))
            spread = 0.0
            if renorm:
                v = v / (v.sum() + 1e-20)
        # expf within 2 ulp of an argument off by half a step of it, at most E + 10 additions
        # and a division, each half a step
        rel[t] = (E + 20 + 2 * spread) * U32
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = v * np.float32(scale)
    flat = ids.reshape(-1)
    order = [i for e in range(E) for i in range(T * k) if flat[i] == e] if T * k <= 4096 else \
        [int(i) for i in np.argsort(np.where(flat < 0, E, flat), kind="stable") if flat[i] >= 0]
    offsets = np.array([(flat[flat >= 0] < e).sum() for e in range(E + 1)], np.int32)
    rows = np.full(T * k, -1, np.int32)
    pos = np.full(T * k, -1, np.int32)
    for slot, i in enumerate(order):
        rows[slot] = i // k
        pos[i] = slot
    return ids, w, offsets, rows, pos.reshape(T, k), rel


# ---------------------------------------------------------------- experts

def dequant(codes, scales, zeros, group):
    """[E][N][K] in binary64 from uint8 codes, float16 scales and packed zero points."""
    E, N, half = codes.shape
    q = np.empty((E, N, 2 * half))
    q[..., 0::2] = codes & 15
    q[..., 1::2] = codes >> 4
    of = np.arange(2 * half) // group
    z = np.full(scales.shape, 8.0)
    if zeros is not None:
        z = np.empty(zeros.shape[:2] + (2 * zeros.shape[2],))
        z[..., 0::2] = zeros & 15
        z[..., 1::2] = zeros >> 4
    return (q - z[..., of]) * scales.astype(np.float64)[..., of]


def spans(offsets, R):
    """(e, first, last) of each expert: offsets clamped to [0, R] and to no less than the one before."""
    o = np.maximum.accumulate(np.clip(offsets.astype(np.int64), 0, R))
    return [(e, int(o[e]), int(o[e + 1])) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def experts(W, x, rows, offsets, y0, swiglu, bf16):
    """y (binary64, y0 where no expert owns the row) and its error bound."""
    R = y0.shape[0]
    K = W.shape[2]
    y, err = y0.astype(np.float64).copy(), np.zeros(y0.shape)
    parts = 1 if bf16 else 3
    # activations: exact (bf16) or two binary16 parts, and the product of the second parts
    # left out; weights: one rounding to binary16 or two parts
    rel = (U16 if bf16 else 2.0 ** -21) + (parts * (K / 16 + 1) + 16) * 2.0 ** -23
    for e, lo, hi in spans(offsets, R):
        xs = np.zeros((hi - lo, K))
        for i, r in enumerate(range(lo, hi)):
            s = r if rows is None else int(rows[r])
            if 0 <= s < x.shape[0]:
                xs[i] = x[s].astype(np.float64)
        v = xs @ W[e].T
        big = np.abs(xs).max(axis=1, keepdims=True)
        # parts below binary16's normal range: half its last step, 2^-25, against the row's
        # largest value scaled to 2^14 and above (activations) or as it is (weights)
        b = rel * (np.abs(xs) @ np.abs(W[e]).T) + 2.0 ** -38 * big * np.abs(W[e]).sum(axis=1)[None, :]
        b = b + 2.0 ** -25 * np.abs(xs).sum(axis=1, keepdims=True)
        if swiglu:
            g, u = v[:, 0::2], v[:, 1::2]
            bg, bu = b[:, 0::2], b[:, 1::2]
            with np.errstate(over="ignore"):
                silu = g / (1.0 + np.exp(-g))
            v = silu * u
            b = 1.1 * bg * (np.abs(u) + bu) + (np.abs(silu) + 1.1 * bg) * bu + 2.0 ** -20 * np.abs(v)
        y[lo:hi] = v
        err[lo:hi] = b + (UBF if bf16 else U32) * (np.abs(v) + b) + 1e-37
    return y, err


# ---------------------------------------------------------------- block norm

def block_norm(y, x, pos, weights, post, gate, alpha, pre, eps, half):
    """out, out_norm (or None) in binary64 and their bounds; half: half a step of the stored type."""
    T, H = x.shape
    y, x = y.astype(np.float64), x.astype(np.float64)
    if pos is None:
        b, s, k = y, np.abs(y), 0
    else:
        k = pos.shape[1]
        b, s = np.zeros((T, H)), np.zeros((T, H))
        for t in range(T):
            for j in range(k):
                if 0 <= pos[t, j] < y.shape[0]:
                    b[t] += float(weights[t, j]) * y[pos[t, j]]
                    s[t] += abs(float(weights[t, j])) * np.abs(y[pos[t, j]])
    eb = (k + 1) * U32 * s                        # k fused multiply-adds

    def rms(v, ev, gamma):
        # the sum of squares in binary32: at most 200 additions in a row, then a division,
        # a root and a reciprocal; its operands off by ev
        m = np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
        with np.errstate(invalid="ignore", divide="ignore"):
            rel = 110 * U32 + np.sqrt((ev * ev).mean(axis=1, keepdims=True)) / m
            out = v / m * gamma
            return out, np.abs(out) * (rel + 3 * U32) + ev / m * np.abs(gamma)

    p, ep = (b, eb) if post is None else rms(b, eb, post.astype(np.float64))
    if gate is not None:
        gate = gate.astype(np.float64)
        ep = ep * np.abs(gate) + U32 * np.abs(gate * p)
        p = gate * p
    out = alpha * x + p
    eo = ep + 2 * U32 * (np.abs(alpha * x) + np.abs(p))
    bound = eo + half * (np.abs(out) + eo) + 1e-37
    if pre is None:
        return out, bound, None, None
    a, ea = rms(out, eo, pre.astype(np.float64))
    return out, bound, a, ea + half * (np.abs(a) + ea) + 1e-37
