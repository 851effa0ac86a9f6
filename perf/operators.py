"""What the mixture-of-experts operators are timed on, and their plain forms.

Four operators, each the feed-forward path of a mixture of experts whose weights are int4
in the MatMulNBits layout (codes [E][N][K/2], binary16 scales [E][N][K/g], 4-bit zero
points [E][N][ceil(K/g/2)]):

  route     router logits -> chosen experts, their weights, and the grouped order of rows
  experts   matrix product of every routed row with its expert's weights (SwiGLU optional)
  norm      weighted sum of a token's expert rows, norm after the block, gate, scaled
            residual, and the norm before the next block
  block     all of them as one call, as a model's layer runs them

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once
at the end) and this package's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a chat: the router of a layer with 64 experts, the smallest call
        dict(name="route 1 token", op="route", T=1, E=64, k=8, score="softmax", renorm=True, bias=False, mask=False),
        # a prompt chunk: sigmoid scores with a balancing bias, padding tokens masked, odd length
        dict(name="route 8191 tokens", op="route", T=8191, E=128, k=8, score="sigmoid", renorm=True, bias=True,
             mask=True),
        # one token, fine-grained experts: gate and up projections, binary32 as the decode GEMVs
        dict(name="gate_up 1 token f32", op="experts", dtype="f32", T=1, E=64, k=8, K=2048, N=2048, group=128,
             sym=False, swiglu=True, gather=True, skew=0.0),
        # sixteen sequences decoding: down projections of the same experts
        dict(name="down 16 tokens f32", op="experts", dtype="f32", T=16, E=64, k=8, K=1024, N=2048, group=32,
             sym=True, swiglu=False, gather=False, skew=0.5),
        # a batch of 48 sequences on eight wide experts of the 8B-class projection shape
        dict(name="gate_up 48 tokens bf16", op="experts", dtype="bf16", T=48, E=8, k=2, K=4096, N=28672, group=128,
             sym=True, swiglu=True, gather=True, skew=0.3),
        # odd sizes of the 0.5B-class shape: 13 groups of 64 in a row, a partial tile of rows, some experts empty
        dict(name="down 333 tokens bf16", op="experts", dtype="bf16", T=333, E=60, k=4, K=832, N=904, group=64,
             sym=False, swiglu=False, gather=False, skew=1.5),
        # a prompt: gate and up projections of fine-grained experts, the largest product
        dict(name="gate_up 4096 tokens bf16", op="experts", dtype="bf16", T=4096, E=64, k=8, K=2048, N=2048, group=64,
             sym=False, swiglu=True, gather=True, skew=0.5),
        # a prompt held in binary32
        dict(name="down 1024 tokens f32", op="experts", dtype="f32", T=1024, E=8, k=2, K=1792, N=4096, group=128,
             sym=False, swiglu=False, gather=False, skew=0.5),
        # one decoded token: eight expert rows summed, norm, layer gate, residual, next norm
        dict(name="norm 1 token bf16", op="norm", dtype="bf16", T=1, H=4096, k=8, post=True, gate="channel", pre=True,
             drop=0.0, alpha=1.0),
        # a prompt with a gate of its own for each token, and some dropped rows
        dict(name="norm 4096 tokens bf16", op="norm", dtype="bf16", T=4096, H=4096, k=8, post=True, gate="token",
             pre=True, drop=0.1, alpha=0.7),
        # one layer's block, eight sequences decoding
        dict(name="block 8 tokens f32", op="block", dtype="f32", T=8, E=64, k=8, H=2048, inner=1024, group=128,
             sym=False, score="softmax", skew=0.5),
        # one layer's block on a prompt
        dict(name="block 2048 tokens bf16", op="block", dtype="bf16", T=2048, E=32, k=4, H=2048, inner=1024, group=64,
             sym=True, score="sigmoid", skew=0.5),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "norm", "block"])
    if op == "route":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 8191), E=E, k=rng.randint(1, min(E, 8)),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5, bias=rng.random() < 0.5,
                    mask=rng.random() < 0.5)
    dtype = rng.choice(["f32", "bf16"])
    group = rng.choice([32, 64, 128])
    if op == "experts":
        T = _log(rng, 1, 4096)
        E = _log(rng, 2, 64)
        k = rng.randint(1, min(E, 8))
        K = group * rng.randint(max(1, 256 // group), 4096 // group)
        N = 2 * rng.randint(64, 2048)
        if T * k * K * N > 10 ** 11:   # no larger than the largest listed product
            T = max(1, 10 ** 11 // (k * K * N))
        return dict(op=op, dtype=dtype, T=T, E=E, k=k, K=K, N=N, group=group, sym=rng.random() < 0.5,
                    swiglu=rng.random() < 0.5, gather=rng.random() < 0.5, skew=round(rng.uniform(0.0, 1.5), 2))
    if op == "norm":
        return dict(op=op, dtype=dtype, T=_log(rng, 1, 2048), H=_log(rng, 64, 8192), k=rng.randint(1, 8),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]), pre=rng.random() < 0.7,
                    drop=rng.choice([0.0, 0.2, 0.9]), alpha=rng.choice([1.0, 0.5]))
    E = rng.choice([8, 16, 32, 47])
    return dict(op=op, dtype=dtype, T=_log(rng, 1, 1024), E=E, k=rng.randint(1, 6), H=128 * rng.randint(2, 16),
                inner=128 * rng.randint(1, 8), group=group, sym=rng.random() < 0.5,
                score=rng.choice(["softmax", "sigmoid"]), skew=round(rng.uniform(0.0, 1.0), 2))


# ------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _weights(g, E, N, K, group, sym):
    """Random int4 experts: uniform codes and zero points, scales uniform on [0.005, 0.02]."""
    nb = K // group
    codes = torch.randint(0, 256, (E, N, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    scales = (0.005 + 0.015 * torch.rand(E, N, nb, device=DEV, generator=g)).half()
    zeros = None
    if not sym:
        zeros = torch.randint(0, 256, (E, N, (nb + 1) // 2), device=DEV, generator=g, dtype=torch.uint8)
        if nb % 2:
            zeros[..., -1] &= 15
    return codes, scales, zeros


def _logits(g, T, E, skew):
    """Router logits: some experts are preferred by all tokens (skew), each token has its own mind."""
    return 1.5 * _normal(g, T, E) + skew * _normal(g, 1, E)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "route":
        s["logits"] = _logits(g, c["T"], c["E"], 0.5)
        s["bias"] = 0.3 * _normal(g, c["E"]) if c["bias"] else None
        s["mask"] = None
        if c["mask"]:
            # padding tokens hold nothing of use, NaN at worst; a few experts are switched off
            s["mask"] = (torch.rand(c["T"], device=DEV, generator=g) < 0.9).to(torch.uint8)
            s["logits"][s["mask"] == 0] = float("nan")
            s["logits"][:, c["E"] // 2] = float("-inf")
        return s
    t = TYPES[c["dtype"]]
    if c["op"] == "experts":
        E, k, T = c["E"], c["k"], c["T"]
        s["codes"], s["scales"], s["zeros"] = _weights(g, E, c["N"], c["K"], c["group"], c["sym"])
        ids = torch.topk(_logits(g, T, E, c["skew"]), k, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        count = torch.bincount(ids, minlength=E)
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
        s["rows"] = (order // k).to(torch.int32) if c["gather"] else None
        s["most"] = int(count.max())   # rows of the busiest expert
        s["x"] = _normal(g, T if c["gather"] else T * k, c["K"]).to(t)
        s["y"] = torch.zeros(T * k, c["N"] // 2 if c["swiglu"] else c["N"], device=DEV, dtype=t)
        return s
    if c["op"] == "norm":
        T, H, k = c["T"], c["H"], c["k"]
        s["y"] = _normal(g, T * k, H).to(t)
        pos = torch.randperm(T * k, device=DEV, generator=g).to(torch.int32).reshape(T, k)
        pos[torch.rand(T, k, device=DEV, generator=g) < c["drop"]] = -1
        s["pos"] = pos
        s["weights"] = torch.softmax(_normal(g, T, k), dim=1)
        s["x"] = (2.0 * _normal(g, T, H)).to(t)
        s["post"] = 0.5 + torch.rand(H, device=DEV, generator=g) if c["post"] else None
        s["pre"] = 0.5 + torch.rand(H, device=DEV, generator=g) if c["pre"] else None
        s["gate"] = None
        if c["gate"] != "none":
            s["gate"] = (1.0 + 0.3 * _normal(g, *((T, H) if c["gate"] == "token" else (H,)))).to(t)
        return s
    T, E, H, inner = c["T"], c["E"], c["H"], c["inner"]
    s["up"] = _weights(g, E, 2 * inner, H, c["group"], c["sym"])
    s["down"] = _weights(g, E, H, inner, c["group"], c["sym"])
    s["logits"] = _logits(g, T, E, c["skew"])
    s["a"] = _normal(g, T, H).to(t)                     # the normed input of the block
    s["x"] = (2.0 * _normal(g, T, H)).to(t)             # the residual stream
    s["post"] = 0.5 + torch.rand(H, device=DEV, generator=g)
    s["pre"] = 0.5 + torch.rand(H, device=DEV, generator=g)
    s["gate"] = (1.0 + 0.3 * _normal(g, H)).to(t)
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_route(logits, k, score, renorm, bias, mask, scale=1.0):
    T, E = logits.shape
    sel = logits + bias if bias is not None else logits
    never = torch.isnan(sel) | (sel == float("-inf"))
    if mask is not None:
        never = never | (mask == 0)[:, None]
    top, ids = torch.sort(sel.masked_fill(never, float("-inf")), dim=1, descending=True, stable=True)
    off = torch.gather(never, 1, ids)[:, :k]
    ids = ids[:, :k]
    raw = logits.masked_fill(torch.isnan(logits), float("-inf"))
    chosen = torch.gather(raw, 1, ids).masked_fill(off, float("-inf")).double()
    if score == "softmax":
        den = chosen if renorm else raw.double()
        high = den.amax(1, keepdim=True)
        high = torch.where(torch.isfinite(high), high, torch.zeros_like(high))
        w = torch.exp(chosen - high) / torch.exp(den - high).sum(1, keepdim=True)
    else:
        w = torch.sigmoid(chosen)
        if renorm:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = torch.where(off, torch.zeros_like(w), w * scale).float()
    ids = ids.masked_fill(off, -1)
    # the grouped order: slots sorted by expert, tokens in order inside one
    flat = torch.where(off, E, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    offsets = (flat[None, :] < torch.arange(E + 1, device=DEV)[:, None]).sum(1)
    slot = torch.arange(T * k, device=DEV)
    rows = torch.where(slot < offsets[E], order // k, -1)
    pos = torch.empty_like(order)
    pos[order] = slot
    pos = pos.reshape(T, k).masked_fill(off, -1)
    return [ids.int(), w, offsets.int(), rows.int(), pos.int()]


def _plain_dequant(codes, scales, zeros, group):
    E, N, half = codes.shape
    q = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(E, N, 2 * half).float()
    q = q.reshape(E, N, -1, group)
    z = torch.full_like(scales, 8.0, dtype=torch.float32)
    if zeros is not None:
        z = torch.stack([zeros & 15, zeros >> 4], dim=-1).reshape(E, N, -1)[..., :scales.shape[2]].float()
    return ((q - z[..., None]) * scales.float()[..., None]).reshape(E, N, 2 * half)


def _plain_experts(w, group, x, rows, offsets, most, swiglu, slots):
    """Every expert's rows padded to `most`, one batched product, the padding dropped."""
    weight = _plain_dequant(*w, group)
    E = weight.shape[0]
    offsets = offsets.long()
    slot = offsets[:-1, None] + torch.arange(most, device=DEV)[None, :]
    used = slot < offsets[1:, None]
    slot = torch.where(used, slot, 0)
    src = rows.long()[slot] if rows is not None else slot
    v = torch.bmm(x.float()[src.clamp_min(0)], weight.transpose(1, 2))
    if swiglu:
        v = v[..., 0::2] * torch.sigmoid(v[..., 0::2]) * v[..., 1::2]
    out = torch.zeros(slots + 1, v.shape[2], device=DEV)
    out[torch.where(used, slot, slots).reshape(-1)] = v.reshape(E * most, -1)
    return out[:slots]


def _plain_rms(v, gamma):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * gamma


def _plain_norm(y, pos, weights, x, post, gate, pre, alpha):
    w = weights.masked_fill(pos < 0, 0.0)
    b = (y.float()[pos.clamp_min(0).long()] * w[..., None]).sum(1)
    if post is not None:
        b = _plain_rms(b, post)
    out = alpha * x.float() + (gate.float() * b if gate is not None else b)
    a = _plain_rms(out, pre) if pre is not None else None
    return [out.to(x.dtype)] + ([a.to(x.dtype)] if a is not None else [])


# ------------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "route":
        return _plain_route(s["logits"], c["k"], c["score"], c["renorm"], s["bias"], s["mask"])
    if c["op"] == "experts":
        v = _plain_experts((s["codes"], s["scales"], s["zeros"]), c["group"], s["x"], s["rows"], s["offsets"],
                           s["most"], c["swiglu"], c["T"] * c["k"])
        return v.to(s["x"].dtype)
    if c["op"] == "norm":
        return _plain_norm(s["y"], s["pos"], s["weights"], s["x"], s["post"], s["gate"], s["pre"], c["alpha"])
    ids, w, offsets, rows, pos = _plain_route(s["logits"], c["k"], c["score"], True, None, None)
    slots = c["T"] * c["k"]
    h = _plain_experts(s["up"], c["group"], s["a"], rows, offsets, c["T"], True, slots)
    y = _plain_experts(s["down"], c["group"], h, None, offsets, c["T"], False, slots)
    return [ids, w] + _plain_norm(y, pos, w, s["x"], s["post"], s["gate"], s["pre"], 1.0)


def _int32(*shape):
    return torch.empty(shape, device=DEV, dtype=torch.int32)


def _run_own(s, c):
    import gemm_decode_gb300 as q4

    if "ws" not in s:   # the workspace that a program keeps for its calls
        T, k = c["T"], c.get("k", 1)
        need = 16
        if c["op"] == "route":
            need = q4.q4moe_route_workspace(T, c["E"], k)
        elif c["op"] == "experts":
            need = q4.q4moe_gemm_workspace(T * k, s["x"].shape[0], c["N"], c["K"], c["E"], s["x"].dtype)
        elif c["op"] == "block":
            need = q4.q4moe_block_workspace(T, c["E"], k, c["H"], c["inner"], s["x"].dtype)
        s["ws"] = torch.empty(need, device=DEV, dtype=torch.uint8)
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        ids, w = _int32(T, k), torch.empty(T, k, device=DEV)
        offsets, rows, pos = _int32(E + 1), _int32(T * k), _int32(T, k)
        q4.q4moe_route_run(s["logits"], ids, w, offsets, rows, pos, s["ws"], bias=s["bias"], token_mask=s["mask"],
                           score=q4.Q4_ROUTE_SIGMOID if c["score"] == "sigmoid" else q4.Q4_ROUTE_SOFTMAX,
                           renormalize=c["renorm"])
        return [ids, w, offsets, rows, pos]
    if c["op"] == "experts":
        q4.q4moe_gemm_run(s["codes"], s["scales"], s["zeros"], s["x"], s["rows"], s["offsets"], s["y"], s["ws"],
                          group=c["group"], epilogue=q4.Q4_EPILOGUE_SWIGLU if c["swiglu"] else q4.Q4_EPILOGUE_NONE)
        return s["y"]
    out = torch.empty_like(s["x"])
    a = torch.empty_like(s["x"]) if s["pre"] is not None else None
    if c["op"] == "norm":
        q4.q4_block_norm_run(s["y"], s["x"], out, pos=s["pos"], weights=s["weights"], post_gamma=s["post"],
                             gate=s["gate"], residual_scale=c["alpha"], pre_gamma=s["pre"], out_norm=a, eps=EPS)
        return [out] + ([a] if a is not None else [])
    ids, w = _int32(c["T"], c["k"]), torch.empty(c["T"], c["k"], device=DEV)
    q4.q4moe_block_run(s["up"], s["down"], s["logits"], s["a"], s["x"], out, a, ids, w, s["ws"], group=c["group"],
                       score=q4.Q4_ROUTE_SIGMOID if c["score"] == "sigmoid" else q4.Q4_ROUTE_SOFTMAX,
                       renormalize=True, post_gamma=s["post"], gate=s["gate"], pre_gamma=s["pre"], eps=EPS)
    return [ids, w, out, a]


# ------------------------------------------------------------------------- the least work

def _size(c):
    return 4 if c["dtype"] == "f32" else 2


def _weight_bytes(N, K, group, sym):
    nb = K // group
    return N * (K // 2 + 2 * nb + (0 if sym else (nb + 1) // 2))


def _active(T, E, k):
    """Experts that at least one of T tokens chooses, were the choices even."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(c):
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        n = 4 * T * E + 16 * T * k + 4 * (E + 1) + (4 * E if c["bias"] else 0) + (T if c["mask"] else 0)
        return {"bytes": n, "flops": 8 * T * E}
    b = _size(c)
    if c["op"] == "experts":
        R, K, N = c["T"] * c["k"], c["K"], c["N"]
        n = _active(c["T"], c["E"], c["k"]) * _weight_bytes(N, K, c["group"], c["sym"])
        n += b * (c["T"] if c["gather"] else R) * K + b * R * (N // 2 if c["swiglu"] else N)
        return {"bytes": n + 4 * (c["E"] + 1) + (4 * R if c["gather"] else 0), "flops": 2 * R * K * N}
    if c["op"] == "norm":
        T, H, k = c["T"], c["H"], c["k"]
        n = b * T * H * (k * (1.0 - c["drop"]) + 2 + (1 if c["gate"] == "token" else 0) + (1 if c["pre"] else 0))
        n += 8 * T * k + 4 * H * (int(c["post"]) + int(c["pre"])) + (b * H if c["gate"] == "channel" else 0)
        return {"bytes": n, "flops": T * H * (2 * k + 8)}
    T, E, k, H, inner = c["T"], c["E"], c["k"], c["H"], c["inner"]
    n = _active(T, E, k) * (_weight_bytes(2 * inner, H, c["group"], c["sym"]) +
                            _weight_bytes(H, inner, c["group"], c["sym"]))
    n += 4 * T * E + 8 * T * k + 4 * b * T * H + (8 + b) * H
    return {"bytes": n, "flops": 2 * T * k * 3 * H * inner}


# ------------------------------------------------------------------------- the definition in 64 bits

def _exact_weight(codes, scales, zeros, e, group):
    """Expert e's matrix, [N][K] in binary64: element k of row n is (q - z) * s of its group."""
    c = codes[e].to(torch.int64)
    N, K = c.shape[0], 2 * c.shape[1]
    q = torch.empty(N, K, dtype=torch.float64, device=DEV)
    q[:, 0::2] = (c % 16).double()
    q[:, 1::2] = torch.div(c, 16, rounding_mode="floor").double()
    of = torch.arange(K, device=DEV) // group
    z = torch.tensor(8.0, dtype=torch.float64, device=DEV)
    if zeros is not None:
        byte = zeros[e].to(torch.int64)[:, of // 2]
        z = torch.where(of % 2 == 0, byte % 16, byte // 16).double()
    return (q - z) * scales[e].double()[:, of]


def _exact_rows(w, group, x, src, ids, swiglu):
    """v[r] = W[ids[r]] x[src[r]] for every slot r in turn of the experts."""
    out = None
    for e in range(w[0].shape[0]):
        at = torch.nonzero(ids == e).reshape(-1)
        if at.numel() == 0:
            continue
        v = x[src[at]].double() @ _exact_weight(*w, e, group).T
        if swiglu:
            v = v[:, 0::2] / (1.0 + torch.exp(-v[:, 0::2])) * v[:, 1::2]
        if out is None:
            out = torch.zeros(ids.numel(), v.shape[1], dtype=torch.float64, device=DEV)
        out[at] = v
    return out


def _exact_weights(logits, k, score, renorm, bias, mask):
    """The experts of each token in order of choice and their weights, token by token on the host."""
    import numpy as np

    l32 = logits.cpu().numpy()
    sel = (l32 + bias.cpu().numpy()).astype(np.float32) if bias is not None else l32
    T, E = l32.shape
    ids, out = np.full((T, k), -1, np.int64), np.zeros((T, k))
    live = np.ones(T, bool) if mask is None else mask.cpu().numpy() != 0
    for t in range(T):
        if not live[t]:
            continue
        order = [int(e) for e in np.lexsort((np.arange(E), -sel[t])) if sel[t, e] > -np.inf][:k]
        if not order:
            continue
        l = l32[t].astype(np.float64)
        if score == "softmax":
            pool = l[order] if renorm else l[~np.isnan(l)]
            v = np.exp(l[order] - pool.max()) / np.exp(pool - pool.max()).sum()
        else:
            v = 1.0 / (1.0 + np.exp(-l[order]))
            if renorm:
                v = v / (v.sum() + 1e-20)
        ids[t, :len(order)], out[t, :len(order)] = order, v
    return torch.from_numpy(ids).to(DEV), torch.from_numpy(out).to(DEV)


def _exact_norm(rows, weights, x, post, gate, pre, alpha):
    """rows [T][k][H] in binary64."""
    b = torch.einsum("tkh,tk->th", rows, weights)
    if post is not None:
        b = b * torch.rsqrt(b.pow(2).mean(1, keepdim=True) + EPS) * post.double()
    out = alpha * x.double() + b * (gate.double() if gate is not None else 1.0)
    if pre is None:
        return [out]
    return [out, out * torch.rsqrt(out.pow(2).mean(1, keepdim=True) + EPS) * pre.double()]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        _, w = _exact_weights(s["logits"], c["k"], c["score"], c["renorm"], s["bias"], s["mask"])
        return [None, w, None, None, None]
    if c["op"] == "experts":
        n = s["offsets"].long()
        ids = torch.repeat_interleave(torch.arange(c["E"], device=DEV), n[1:] - n[:-1])
        src = s["rows"].long() if s["rows"] is not None else torch.arange(ids.numel(), device=DEV)
        return _exact_rows((s["codes"], s["scales"], s["zeros"]), c["group"], s["x"], src, ids, c["swiglu"])
    if c["op"] == "norm":
        live = s["pos"] >= 0
        out = []
        for part in torch.split(torch.arange(c["T"], device=DEV), 1024):   # binary64 rows of 1024 tokens at a time
            rows = s["y"][s["pos"][part].clamp_min(0).long()].double()
            gate = s["gate"][part] if c["gate"] == "token" else s["gate"]
            out.append(_exact_norm(rows, s["weights"][part].double() * live[part], s["x"][part], s["post"], gate,
                                   s["pre"], c["alpha"]))
        return [torch.cat(p) for p in zip(*out)]
    ids, w = _exact_weights(s["logits"], c["k"], c["score"], True, None, None)
    T, k = ids.shape
    src = torch.arange(T * k, device=DEV) // k
    h = _exact_rows(s["up"], c["group"], s["a"], src, ids.reshape(-1), True)
    y = _exact_rows(s["down"], c["group"], h, torch.arange(T * k, device=DEV), ids.reshape(-1), False)
    return [None, w] + _exact_norm(y.reshape(T, k, -1), w, s["x"], s["post"], s["gate"], s["pre"], 1.0)
