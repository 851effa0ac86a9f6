"""Error bounds of the expert products, from the arithmetic of each of the two kernels.

Half a step of a rounding, relative to the value: binary32 2^-24, binary16 2^-11, bfloat16
2^-8.

Activations.  A row of x is scaled by a power of two so that its largest element lies in
[2^14, 2^15), and held in binary16: one part (bfloat16, 8 bits: exact down to binary16's last
step) or two (binary32: each part half a step, 2^-22 together).  Below, binary16's step is
2^-24 whatever the value: half of it, 2^-25, against 2^14 for the row's largest element.

Few rows per expert.  Weights are whole numbers, exact.  The tensor core adds up one group, 16
products at a time, and may cut instead of round: 2^-23 of what it adds, g / 16 times.  Then
two binary32 roundings per group (the parts of x, the sum), one per part joined.

Many rows.  Weights are rounded to binary16 (half of its last step, 2^-25, for tiny ones); one
sum over K, 16 products at a time.
"""
import numpy as np

U32, U16, UBF = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


def is_few(R, E, bf16):
    """Whether the kernel for few rows per expert serves the call."""
    return not bf16 or R <= 24 * E


def spans(offsets, R):
    o = np.maximum.accumulate(np.clip(offsets.astype(np.int64), 0, R))
    return [(e, int(o[e]), int(o[e + 1])) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def product(xs, W, group, few, bf16):
    """v = xs W^T in binary64 and its bound before the output's rounding."""
    K = W.shape[1]
    v, S = xs @ W.T, np.abs(xs) @ np.abs(W).T
    lost = (0.0 if bf16 else 2.0 ** -22) * np.abs(xs)
    lost = lost + 2.0 ** -39 * np.abs(xs).max(axis=1, keepdims=True) + 2.0 ** -151 * (not bf16)
    b = lost @ np.abs(W).T
    joined = K / 128
    if few:
        b = b + (group / 16 * 2.0 ** -23 * (1 + 2.0 ** -10) + (2 * K / group + joined + 3) * U32) * S
    else:
        b = b + (U16 * (1 + 2.0 ** -10) + (K / 16 + 1) * 2.0 ** -23 + (joined + 3) * U32) * S
        b = b + 2.0 ** -25 * np.abs(xs).sum(axis=1, keepdims=True)
    return v, b


def experts(W, x, rows, offsets, y0, swiglu, bf16, group):
    """y (binary64, y0 where no expert owns the row) and its bound."""
    R, E, K = y0.shape[0], W.shape[0], W.shape[2]
    y, err = y0.astype(np.float64).copy(), np.zeros(y0.shape)
    for e, lo, hi in spans(offsets, R):
        xs = np.zeros((hi - lo, K))
        for i, r in enumerate(range(lo, hi)):
            s = r if rows is None else int(rows[r])
            if 0 <= s < x.shape[0]:
                xs[i] = x[s].astype(np.float64)
        v, b = product(xs, W[e], group, is_few(R, E, bf16), bf16)
        if swiglu:
            g, u, bg, bu = v[:, 0::2], v[:, 1::2], b[:, 0::2], b[:, 1::2]
            with np.errstate(over="ignore"):
                silu = g / (1.0 + np.exp(-g))
            # silu's slope is at most 1.1; the exponential and the division: 8 steps of binary32,
            # with the fast ones of the bfloat16 form 2^-20
            v = silu * u
            b = 1.1 * bg * (np.abs(u) + bu) + np.abs(silu) * bu + (2.0 ** -20 if bf16 else 8 * U32) * np.abs(v)
        y[lo:hi] = v
        err[lo:hi] = b + (UBF if bf16 else U32) * (np.abs(v) + b) + 1e-37
    return y, err


def two_norm(K, group):
    """Relative error, 2-norm over many outputs of random weights and activations, of the
    kernel for few rows in binary32.  x: 2^-22.  A sum of 16 i products has a size of
    sqrt(16 i); each of the g / 16 additions of a group cuts up to 2^-25 of it (measured on
    this tensor core: 2e-8 of the sum), all in one direction, so the K / g groups add up;
    the result's size is sqrt(K).  The K / g binary32 additions round either way."""
    cuts = K / group * sum(4 * np.sqrt(i + 1) for i in range(group // 16)) / np.sqrt(K)
    return 2.0 ** -22 + cuts * 2.0 ** -25 + np.sqrt(K / group) * U32


# Outputs of the bfloat16 kernel for few rows that are not the exact value's own rounding: an
# error of at most two_norm (1e-6 of the outputs' usual size) against bfloat16 steps of 2^-8 to
# 2^-7 of each output, small outputs having small steps: 1e-6 x 2^8 x about 5.  Binary16
# weights (2e-4) misround one output in ten.
MISROUNDED = 5e-3
