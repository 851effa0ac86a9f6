"""Binary64 forms of the calls for several continuations of one prompt, and the error bounds of
their kernels.  numpy and torch on the CPU; nothing of the library.

Half a step of a rounding, relative to the value: binary32 2^-24, binary16 2^-11 (and 2^-25
absolute below 2^-14), bfloat16 2^-8."""
import math

import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rounding(y, dtype):
    """What rounding y to a type may move it by."""
    return HALF_STEP[dtype] * y.abs() + TINY[dtype]


def within(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((off / bound.clamp_min(1e-300)).nan_to_num(1e9).max()):.3g} of the bound, first at "
                           f"{tuple(int(i) for i in bad.nonzero()[0])}")


# ------------------------------------------------------------------------- rotary positions

def rope(x, gamma, positions, inv_freq, half_layout, scale, eps):
    """(y, bound before the output's rounding) of heads x [T, H, D]."""
    x = x.double().cpu()
    D, rot = x.shape[-1], 2 * inv_freq.numel()
    u = x
    if gamma is not None:
        u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double().cpu()
    turns = positions.double().cpu()[:, None] * (inv_freq.double().cpu() / (2 * math.pi))
    angle = 2 * math.pi * (turns - turns.round())   # binary64 keeps 2^-53 of 2^31 turns: 2^-22 of one at worst
    c, s = (scale * f(angle)[:, None, :] for f in (torch.cos, torch.sin))
    i = torch.arange(rot // 2)
    a, b = (i, i + rot // 2) if half_layout else (2 * i, 2 * i + 1)
    y = u.clone()
    y[..., a] = c * u[..., a] - s * u[..., b]
    y[..., b] = s * u[..., a] + c * u[..., b]
    # The norm: a sum of D squares in any order (D 2^-24 at most, halved by the root), a root, a
    # division and two products.  Cosines and sines: within 2^-21 of the scale; two products, a sum.
    own = ((D / 2 + 6) * U32 if gamma is not None else 0.0) * u.abs()
    bound = own.clone()
    both = u[..., a].abs() + u[..., b].abs()
    for j in (a, b):
        bound[..., j] = abs(scale) * ((own[..., a] + own[..., b]) + (2.0 ** -21 + 4 * U32) * both)
    return y, bound


# ------------------------------------------------------------------------- attention

def keys_of(cache, table, n, head):
    """Rows [0, n) of a kv head of the sequence a page table names; pages outside the pool are zeros."""
    pages, _, page, D = cache.shape
    out = torch.zeros(n, D, dtype=torch.float64)
    for j in range((n + page - 1) // page):
        p, m = int(table[j]), min(page, n - j * page)
        if 0 <= p < pages:
            out[j * page:j * page + m] = cache[p, head, :m].double()
    return out


def spans(offsets, groups, S):
    if offsets is None:
        return [(0, S)]
    o, last = [], 0
    for v in offsets.tolist():
        last = max(last, min(max(v, 0), S))
        o.append(last)
    return [(o[g], o[g + 1]) for g in range(groups)]


def attention(q, k_cache, v_cache, offsets, shared_pages, shared_lens, limits, own_pages, own_lens, scale, type16):
    """(o, lse, bound of o before the output's rounding, bound of lse)."""
    q, kc, vc = q.double().cpu(), k_cache.cpu(), v_cache.cpu()
    S, Hq, D = q.shape
    page, G = kc.shape[2], Hq // kc.shape[1]
    groups = shared_lens.numel() if shared_lens is not None else 0
    of = [-1] * S
    for g, (a, b) in enumerate(spans(offsets, groups, S) if groups else []):
        for s in range(a, b):
            of[s] = g
    clamp = lambda n, table: max(0, min(int(n), table.shape[1] * page))  # noqa: E731
    o, lse = torch.zeros(S, Hq, D, dtype=torch.float64), torch.full((S, Hq), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    U = HALF_STEP[type16]
    for h in range(kc.shape[1]):
        held = {}
        for g in range(groups):
            n = clamp(shared_lens[g], shared_pages)
            held[g] = keys_of(kc, shared_pages[g], n, h), keys_of(vc, shared_pages[g], n, h)
        for s in range(S):
            ks, vs = [torch.zeros(0, D, dtype=torch.float64)], [torch.zeros(0, D, dtype=torch.float64)]
            if of[s] >= 0:
                k, v = held[of[s]]
                n = k.shape[0] if limits is None else max(0, min(k.shape[0], int(limits[s])))
                ks.append(k[:n]), vs.append(v[:n])
            if own_lens is not None:
                n = clamp(own_lens[s], own_pages)
                ks.append(keys_of(kc, own_pages[s], n, h)), vs.append(keys_of(vc, own_pages[s], n, h))
            k, v = torch.cat(ks), torch.cat(vs)
            if k.shape[0] == 0:
                continue
            r = slice(h * G, (h + 1) * G)
            x = scale * (q[s, r] @ k.T)
            high = x.amax(1, keepdim=True)
            p = torch.exp(x - high)
            l = p.sum(1, keepdim=True)
            o[s, r] = p @ v / l
            lse[s, r] = (high + torch.log(l))[:, 0]
            # A score: D products summed 16 at a time, each step cut at 2^-23 of what it adds, then
            # scaled (to a power of two) and subtracted: D / 16 + 6 steps of binary32 on |scale| |q| |k|.
            # The exponential doubles as much again; joining parts adds a few steps to each weight.
            dx = (abs(scale) * (q[s, r].abs() @ k.abs().T).amax(1, keepdim=True) * (D / 16 + 6) +
                  2 * x.abs().amax(1, keepdim=True) + 16) * 2.0 ** -23
            steps = (k.shape[0] / 16 + 64) * 2.0 ** -23          # sums over the keys
            w = p @ v.abs() / l
            tiny = (TINY[type16] * v.abs().sum(0) / l) if type16 is torch.float16 else 0.0
            bo[s, r] = w * (U + 2 * (torch.exp(2 * dx) - 1) + 2 * steps) + tiny
            bl[s, r] = (2 * dx + 2 * steps + 2.0 ** -22 * lse[s, r, None].abs())[:, 0]
    return o, lse, bo, bl


# ------------------------------------------------------------------------- beams

def beam_step(logits, scores, finished, K, eos):
    """(tokens, parents, scores, finished) by the definition: candidates sorted by score, beam, token."""
    groups, W = scores.shape
    l = logits.double().cpu().reshape(groups, W, -1)
    l = torch.where(torch.isfinite(l), l, -math.inf)
    V = l.shape[2]
    tokens, parents = torch.full((groups, K), -1), torch.full((groups, K), -1)
    best, fin = torch.full((groups, K), -math.inf, dtype=torch.float64), torch.zeros(groups, K, dtype=torch.uint8)
    for g in range(groups):
        cum = scores[g].double().cpu()
        s = torch.full((W, V), -math.inf, dtype=torch.float64)
        for w in range(W):
            if not math.isfinite(cum[w]):
                continue
            if finished is not None and finished[g, w]:
                s[w, eos] = cum[w]
            elif torch.isfinite(l[g, w]).any():
                high = l[g, w].max()
                s[w] = cum[w] + (l[g, w] - (high + torch.log(torch.exp(l[g, w] - high).sum())))
        top, at = torch.sort(s.reshape(-1), descending=True, stable=True)
        for j in range(min(K, W * V)):
            if top[j] > -math.inf:
                tokens[g, j], parents[g, j], best[g, j] = at[j] % V, at[j] // V, top[j]
                fin[g, j] = int(at[j] % V) == eos
    return tokens, parents, best, fin


def reorder(tables, lens, parents, spare, pool):
    """(out_tables, out_spare, pool) after a beam step."""
    groups, W = parents.shape
    planes, pages, heads, page, D = pool.shape
    new, left, out = tables.clone(), spare.clone(), pool.clone()
    most = tables.shape[1]
    for g in range(groups):
        n = max(0, min(int(lens[g]), most * page))
        f, r = n // page, n % page
        for w in range(W):
            i, p = g * W + w, int(parents[g, w])
            p = g * W + (p if 0 <= p < W else w)
            new[i, :f] = tables[p, :f]
            if r > 0 and p != i:
                new[i, f], left[i] = spare[i], tables[i, f]
                src, dst = int(tables[p, f]), int(spare[i])
                if 0 <= src < pages and 0 <= dst < pages:
                    out[:, dst, :, :r] = pool[:, src, :, :r]
    return new, left, out
