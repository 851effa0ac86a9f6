"""What the operators of decoding several continuations of one prompt are timed on, and their
plain forms.

Four operators, the attention side of a layer next to the int4 products and what follows the
LM head, as a batch that shares prompts or a beam search runs them:

  rope       norm of the queries and keys of each head, rotary positions (half or interleaved
             pairs, the whole head or its first features), and the new keys and values put
             into a paged cache
  attention  attention over that cache: a segment shared by a group of sequences, read once
             for all of them, then each sequence's own segment; with a limit for each query
             also the causal attention of a prompt
  beam       log-softmax of every beam's logits, the best continuations over beams and
             vocabulary, and their parents
  reorder    the page tables and the unfinished pages of all layers follow the parents

The paged cache is two pools, keys and values, [pages][kv heads][tokens of a page][features];
a page table names the pages of a sequence.  `own` chooses between the plain form (elementary
torch operations in 32 bits, rounded once at the end) and this package's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # four beams, one step: projections of the decode GEMV (binary32), the 8B-class heads; the smallest call
        dict(name="rope 4 tokens f32", op="rope", T=4, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="f32",
             cache="bf16", norm=True, page=16, start=1000, drop=0.0),
        # a prompt chunk far into a long context, the same heads
        dict(name="rope 4096 tokens bf16", op="rope", T=4096, Hq=32, Hkv=8, D=128, rot=128, layout="half",
             dtype="bf16", cache="bf16", norm=True, page=64, start=120000, drop=0.0),
        # the 0.5B-class heads: seven query heads to a kv head, half of the head rotated in interleaved pairs,
        # no norm, an odd length with padding tokens
        dict(name="rope 777 tokens f32", op="rope", T=777, Hq=14, Hkv=2, D=64, rot=32, layout="interleaved",
             dtype="f32", cache="f16", norm=False, page=32, start=0, drop=0.1),
        # four beams of a short prompt, a few tokens in: latency
        dict(name="attention 4 beams", op="attention", Hq=32, Hkv=8, D=128, cache="bf16", page=16, groups=1, most=4,
             least=4, shared=1000, ragged=0.0, own=20, causal=False),
        # 16 prompts of 8 beams each, prompts and continuations of different lengths, 0.5B-class heads
        dict(name="attention 16 prompts 8 beams f16", op="attention", Hq=14, Hkv=2, D=64, cache="f16", page=32,
             groups=16, most=8, least=8, shared=2048, ragged=0.5, own=100, causal=False),
        # a batch behind one system prompt, own parts of up to 1024 tokens
        dict(name="attention 64 sequences one prefix", op="attention", Hq=32, Hkv=8, D=128, cache="bf16", page=16,
             groups=1, most=64, least=64, shared=8192, ragged=0.5, own=1024, causal=False),
        # the same kind of batch at the far end: many sequences, a long document
        dict(name="attention 256 sequences long prefix", op="attention", Hq=32, Hkv=8, D=128, cache="bf16", page=64,
             groups=1, most=256, least=256, shared=32768, ragged=0.3, own=256, causal=False),
        # a prompt of 4096 tokens against itself: causal limits, no own segments
        dict(name="attention prompt 4096 causal", op="attention", Hq=32, Hkv=8, D=128, cache="bf16", page=64,
             groups=1, most=4096, least=4096, shared=4096, ragged=0.0, own=0, causal=True),
        # one prompt, four beams: the 0.5B-class vocabulary
        dict(name="beam 1 x 4", op="beam", groups=1, W=4, K=4, V=151936, finished=0.0, banned=0.0),
        # 16 prompts of 8 beams, the 8B-class vocabulary, some beams finished, some tokens banned
        dict(name="beam 16 x 8", op="beam", groups=16, W=8, K=8, V=128256, finished=0.1, banned=0.01),
        # one prompt, four beams, 24 layers of the 0.5B class
        dict(name="reorder 1 x 4", op="reorder", groups=1, W=4, planes=48, Hkv=2, D=64, cache="bf16", page=16,
             maxp=64, length=200),
        # 16 prompts of 8 beams, 32 layers of the 8B class, odd lengths
        dict(name="reorder 16 x 8", op="reorder", groups=16, W=8, planes=64, Hkv=8, D=128, cache="bf16", page=16,
             maxp=128, length=1500),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "attention", "beam", "reorder"])
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    cache, page = rng.choice(["bf16", "bf16", "f16"]), rng.choice([16, 32, 64, 128])
    if op == "rope":
        Hq = Hq if Hq <= 32 else Hkv
        return dict(op=op, T=_log(rng, 1, 4096), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 16, 24]),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["f32", "bf16"]), cache=cache,
                    norm=rng.random() < 0.5, page=page, start=_log(rng, 1, 10 ** 6), drop=rng.choice([0.0, 0.2]))
    if op == "attention":
        if rng.random() < 0.25:   # prompts
            groups = rng.randint(1, 4)
            most = _log(rng, 2, 4096 // groups)
            shared, mine, causal = most + rng.choice([0, _log(rng, 1, 1024)]), 0, True
        else:
            groups = _log(rng, 1, 16)
            most = _log(rng, 1, 256 // groups)
            shared, mine, causal = _log(rng, 1, 32768), rng.choice([0, _log(rng, 1, 1024)]), False
        # no larger than the largest listed: the plain form holds a score for every pair
        while groups * most * Hq * (shared + mine) > 256 * 32 * 33000:
            shared, most = max(1, shared // 2) if not causal else most // 2 + shared - most, max(1, most // 2)
        return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, cache=cache, page=page, groups=groups, most=most,
                    least=most if causal else rng.randint(max(1, most // 2), most), shared=shared,
                    ragged=0.0 if causal else round(rng.uniform(0.0, 1.0), 2), own=mine, causal=causal)
    if op == "beam":
        groups, W = _log(rng, 1, 16), rng.randint(1, 16)
        V = _log(rng, 1000, 152000)
        while groups * W * V > 128 * 128256:
            groups = max(1, groups // 2)
        return dict(op=op, groups=groups, W=W, K=rng.choice([W, W, min(32, 2 * W)]), V=V,
                    finished=rng.choice([0.0, 0.2]), banned=rng.choice([0.0, 0.01, 0.5]))
    maxp = rng.randint(2, 128)
    groups, W, planes = _log(rng, 1, 16), rng.randint(1, 8), 2 * rng.randint(1, 32)
    page = rng.choice([16, 32])
    while groups * W * planes * Hkv * D * page > 16 * 8 * 64 * 8 * 128 * 16:
        planes = max(2, planes // 4 * 2)
        groups = max(1, groups // 2)
    return dict(op=op, groups=groups, W=W, planes=planes, Hkv=Hkv, D=D, cache=cache, page=page, maxp=maxp,
                length=rng.randint(0, maxp * page - 1))


# ------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _whole(g, low, high, *shape):
    """Whole numbers of [low, high]."""
    return torch.randint(low, high + 1, shape, device=DEV, generator=g)


def _paged(g, pages, lens, page):
    """Page tables [len(lens)][most pages] of sequences of these lengths (at most `lens.max()`), from `pages`,
    a shuffled list of free pages; entries behind the last page of a sequence are -1."""
    need = (lens + page - 1) // page
    first = need.cumsum(0) - need
    most = max(1, int(need.max()))
    j = torch.arange(most, device=DEV)
    at = first[:, None] + j[None, :]
    table = pages[at.clamp_max(pages.numel() - 1)]
    return torch.where(j[None, :] < need[:, None], table, -1).to(torch.int32), pages[int(need.sum()):]


def _members(c):
    """Sequences of each group: between `least` and `most`, the last group the largest."""
    n = [c["least"] + 7 * i % (c["most"] - c["least"] + 1) for i in range(c["groups"])]
    return n[:-1] + [c["most"]]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "rope":
        T, Hq, Hkv, D, t16 = c["T"], c["Hq"], c["Hkv"], c["D"], TYPES[c["cache"]]
        # one row holds a token's queries, keys and values, as one product makes them
        qkv = (2.0 * _normal(g, T, (Hq + 2 * Hkv) * D)).to(TYPES[c["dtype"]])
        s["qkv"] = qkv
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["positions"] = (c["start"] + torch.arange(T, device=DEV) + 3 * int(seed) % 64).to(torch.int32)
        i = torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = (500000.0 ** (-i / c["rot"])).float()
        s["q_gamma"] = 0.5 + torch.rand(D, device=DEV, generator=g) if c["norm"] else None
        s["k_gamma"] = 0.5 + torch.rand(D, device=DEV, generator=g) if c["norm"] else None
        used = (T + c["page"] - 1) // c["page"]
        pages = torch.randperm(used + 2, device=DEV, generator=g)[:used]
        t = torch.arange(T, device=DEV)
        slots = pages[t // c["page"]] * c["page"] + t % c["page"]
        slots[torch.rand(T, device=DEV, generator=g) < c["drop"]] = -1   # padding tokens
        s["slots"] = slots.to(torch.int32)
        s["q_out"] = torch.zeros(T, Hq, D, device=DEV, dtype=t16)
        s["k_cache"] = _normal(g, used + 2, Hkv, c["page"], D).to(t16)
        s["v_cache"] = _normal(g, used + 2, Hkv, c["page"], D).to(t16)
        return s
    if c["op"] == "attention":
        Hkv, D, page, t16 = c["Hkv"], c["D"], c["page"], TYPES[c["cache"]]
        n = torch.tensor(_members(c), device=DEV)
        s["group_offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        S = int(n.sum())
        cut = lambda most, count: (most - (most * c["ragged"] * torch.rand(count, device=DEV, generator=g)).long())  # noqa: E731
        shared_lens = cut(c["shared"], c["groups"])
        own_lens = cut(c["own"], S) if c["own"] else None
        total = int(((shared_lens + page - 1) // page).sum()) + 1
        if own_lens is not None:
            total += int(((own_lens + page - 1) // page).sum())
        free = torch.randperm(total, device=DEV, generator=g)
        s["shared_pages"], free = _paged(g, free, shared_lens, page)
        s["shared_lens"] = shared_lens.to(torch.int32)
        s["own_pages"] = s["own_lens"] = s["limits"] = None
        if own_lens is not None:
            s["own_pages"], free = _paged(g, free, own_lens, page)
            s["own_lens"] = own_lens.to(torch.int32)
        if c["causal"]:   # token i of a prompt's last n sees the tokens before them, and itself
            i = torch.arange(S, device=DEV)
            of = torch.searchsorted(s["group_offsets"][1:].long(), i, right=True)
            s["limits"] = (shared_lens[of] - n[of] + i - s["group_offsets"][of] + 1).to(torch.int32)
        s["q"] = (1.5 * _normal(g, S, c["Hq"], D)).to(t16)
        s["k_cache"] = _normal(g, total, Hkv, page, D).to(t16)
        s["v_cache"] = _normal(g, total, Hkv, page, D).to(t16)
        s["out"] = torch.zeros(S, c["Hq"], D, device=DEV, dtype=t16)
        return s
    if c["op"] == "beam":
        S = c["groups"] * c["W"]
        s["logits"] = 2.5 * _normal(g, S, c["V"])
        s["logits"][torch.rand(S, c["V"], device=DEV, generator=g) < c["banned"]] = float("-inf")
        s["scores"] = -20.0 * torch.rand(c["groups"], c["W"], device=DEV, generator=g)
        s["eos"] = c["V"] // 2
        s["finished"] = (torch.rand(c["groups"], c["W"], device=DEV, generator=g) < c["finished"]).to(torch.uint8)
        return s
    groups, W, page, maxp = c["groups"], c["W"], c["page"], c["maxp"]
    S = groups * W
    s["lens"] = (c["length"] - _whole(g, 0, min(c["length"], 40), groups)).clamp_min(0).to(torch.int32)
    s["parents"] = _whole(g, 0, W - 1, groups, W).to(torch.int32)
    # the pages being written (one for each beam) and the spare ones are in the pool; the full pages before them
    # are named by the tables only, and nothing here reads them
    order = torch.randperm(2 * S, device=DEV, generator=g).to(torch.int32)
    s["tables"] = _whole(g, 0, 2 * S - 1, S, maxp).to(torch.int32)
    at = (s["lens"].long() // page).repeat_interleave(W)
    s["tables"][torch.arange(S, device=DEV), at] = order[:S]
    s["spare"] = order[S:].clone()
    s["pool"] = _normal(g, c["planes"], 2 * S, c["Hkv"], page, c["D"]).to(TYPES[c["cache"]])
    s["out_tables"], s["out_spare"] = torch.zeros_like(s["tables"]), torch.zeros_like(s["spare"])
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_rope(x, gamma, cos, sin, layout):
    x = x.float()
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    rest = x[..., 2 * half:]
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)
    a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2), rest], dim=-1)


def _plain_append(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    t16 = s["q_out"].dtype
    s["q_out"].copy_(_plain_rope(s["q"], s["q_gamma"], cos, sin, c["layout"]).to(t16))
    kept = torch.nonzero(s["slots"] >= 0).reshape(-1)
    slot = s["slots"][kept].long()
    k = _plain_rope(s["k"], s["k_gamma"], cos, sin, c["layout"]).to(t16)
    s["k_cache"][slot // c["page"], :, slot % c["page"]] = k[kept]
    s["v_cache"][slot // c["page"], :, slot % c["page"]] = s["v"].float().to(t16)[kept]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_gather(cache, table, most):
    """The first `most` rows of each sequence of a page table, [sequences][kv heads][most][D], in 32 bits."""
    rows = cache[table.clamp_min(0).long()]                      # [n][pages][Hkv][page][D]
    rows = rows.transpose(1, 2).flatten(2, 3)[:, :, :most].float()
    return rows


def _plain_attention(s):
    c = s["case"]
    S, Hq, D = s["q"].shape
    Hkv, G = c["Hkv"], Hq // c["Hkv"]
    q = s["q"].float().reshape(S, Hkv, G, D) / math.sqrt(D)
    first = s["group_offsets"].long()
    i = torch.arange(S, device=DEV)
    of = torch.searchsorted(first[1:], i, right=True)            # the group of each query, and its place there
    place = i - first[of]
    # queries padded to the largest group: [groups][Hkv][most * G][D]
    qg = torch.zeros(c["groups"], c["most"], Hkv, G, D, device=DEV)
    qg[of, place] = q
    qg = qg.transpose(1, 2).flatten(2, 3)
    k, v = (_plain_gather(s[n], s["shared_pages"], c["shared"]) for n in ("k_cache", "v_cache"))
    limit = s["shared_lens"].long()[of]
    if s["limits"] is not None:
        limit = torch.minimum(limit, s["limits"].long())
    lim = torch.zeros(c["groups"], c["most"], device=DEV, dtype=torch.long)
    lim[of, place] = limit
    seen = torch.arange(k.shape[2], device=DEV) < lim[..., None]                 # [groups][most][keys]
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    scores = torch.matmul(qg, k.transpose(2, 3)).masked_fill_(~seen, float("-inf"))
    high = scores.amax(3).reshape(c["groups"], Hkv, c["most"], G).transpose(1, 2)[of, place]   # [S][Hkv][G]
    if s["own_lens"] is not None:
        ko, vo = (_plain_gather(s[n], s["own_pages"], c["own"]) for n in ("k_cache", "v_cache"))
        mine = torch.matmul(q, ko.transpose(2, 3))
        live = torch.arange(ko.shape[2], device=DEV) < s["own_lens"].long()[:, None]
        mine = mine.masked_fill(~live[:, None, None], float("-inf"))
        high = torch.maximum(high, mine.amax(3))
    high = torch.where(torch.isfinite(high), high, torch.zeros_like(high))
    hg = torch.zeros(c["groups"], c["most"], Hkv, G, device=DEV)
    hg[of, place] = high
    p = torch.exp(scores - hg.transpose(1, 2).flatten(2, 3)[..., None])
    total = torch.matmul(p, v).reshape(c["groups"], Hkv, c["most"], G, D).transpose(1, 2)[of, place]
    count = p.sum(3).reshape(c["groups"], Hkv, c["most"], G).transpose(1, 2)[of, place]
    if s["own_lens"] is not None:
        p = torch.exp(mine - high[..., None])
        total = total + torch.matmul(p, vo)
        count = count + p.sum(3)
    out = torch.where(count[..., None] > 0, total / count[..., None], torch.zeros_like(total))
    return out.reshape(S, Hq, D).to(s["q"].dtype)


def _plain_beam(s):
    c = s["case"]
    groups, W, K, V = c["groups"], c["W"], c["K"], c["V"]
    l = s["logits"].double()
    high = l.amax(1, keepdim=True)
    lse = high + torch.log(torch.exp(l - high).sum(1, keepdim=True))
    score = (s["scores"].double().reshape(-1, 1) + (l - lse)).reshape(groups, W, V)
    done = s["finished"] != 0
    # a finished beam goes on as it is: its only continuation is the end token, at no cost
    score = score.masked_fill(done[..., None], float("-inf"))
    score[..., s["eos"]] = torch.where(done, s["scores"].double(), score[..., s["eos"]])
    best, at = torch.sort(score.reshape(groups, W * V), dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    none = best == float("-inf")
    tokens, parents = (at % V).masked_fill(none, -1), (at // V).masked_fill(none, -1)
    finished = (tokens == s["eos"]) & ~none
    return [tokens.int(), parents.int(), best.float(), finished.to(torch.uint8)]


def _plain_reorder(s):
    c = s["case"]
    groups, W, page, maxp = c["groups"], c["W"], c["page"], c["maxp"]
    S = groups * W
    i = torch.arange(S, device=DEV)
    parent = (s["parents"].long() + W * torch.arange(groups, device=DEV)[:, None]).reshape(S)
    n = s["lens"].long().repeat_interleave(W)
    full, rest = n // page, n % page
    moved = (parent != i) & (rest > 0)
    j = torch.arange(maxp, device=DEV)
    tables = torch.where(j[None, :] < full[:, None], s["tables"][parent], s["tables"])
    mine = s["tables"][i, full]
    tables[i, full] = torch.where(moved, s["spare"], mine)
    s["out_tables"].copy_(tables)
    s["out_spare"].copy_(torch.where(moved, mine, s["spare"]))
    m = torch.nonzero(moved).reshape(-1)
    src, dst = s["tables"][parent[m], full[m]].long(), s["spare"][m].long()
    row = torch.arange(page, device=DEV)
    rows = torch.where(row[None, :, None] < rest[m][:, None, None, None], s["pool"][:, src], s["pool"][:, dst])
    s["pool"][:, dst] = rows
    return [s["out_tables"], s["out_spare"], s["pool"]]


# ------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, s["case"])
    if op == "rope":
        return _plain_append(s)
    if op == "attention":
        return _plain_attention(s)
    return _plain_beam(s) if op == "beam" else _plain_reorder(s)


def _run_own(s, c):
    import gemm_decode_gb300 as q4

    if c["op"] == "rope":
        q4.q4_rope_append_run(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["q_out"], s["k_cache"],
                              s["v_cache"], slots=s["slots"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS,
                              layout=q4.Q4_ROPE_HALF if c["layout"] == "half" else q4.Q4_ROPE_INTERLEAVED)
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if c["op"] == "attention":
        if "ws" not in s:   # the workspace that a program keeps for its calls
            S, Hq, D = s["q"].shape
            need = q4.q4_prefix_attn_workspace(S, c["groups"], Hq, c["Hkv"], D)
            s["ws"] = torch.empty(need, device=DEV, dtype=torch.uint8)
        q4.q4_prefix_attn_run(s["q"], s["k_cache"], s["v_cache"], s["out"], s["ws"],
                              group_offsets=s["group_offsets"], shared_pages=s["shared_pages"],
                              shared_lens=s["shared_lens"], limits=s["limits"], own_pages=s["own_pages"],
                              own_lens=s["own_lens"])
        return s["out"]
    if c["op"] == "beam":
        groups, W, K, V = c["groups"], c["W"], c["K"], c["V"]
        if "ws" not in s:
            s["ws"] = torch.empty(q4.q4_beam_step_workspace(groups, W, K, V), device=DEV, dtype=torch.uint8)
        tokens, parents = (torch.empty(groups, K, device=DEV, dtype=torch.int32) for _ in range(2))
        scores = torch.empty(groups, K, device=DEV)
        finished = torch.empty(groups, K, device=DEV, dtype=torch.uint8)
        q4.q4_beam_step_run(s["logits"], s["scores"], tokens, parents, scores, s["ws"], finished=s["finished"],
                            out_finished=finished, eos=s["eos"])
        return [tokens, parents, scores, finished]
    q4.q4_beam_reorder_run(s["tables"], s["lens"], s["parents"], s["spare"], s["out_tables"], s["out_spare"], s["pool"])
    return [s["out_tables"], s["out_spare"], s["pool"]]


# ------------------------------------------------------------------------- the least work

def _attention_rows(c):
    """Queries, and keys that are read: expected ones where the lengths are drawn."""
    S = sum(_members(c))
    mean = 1.0 - c["ragged"] / 2
    return S, c["groups"] * c["shared"] * mean, S * c["own"] * mean


def work(c):
    if c["op"] == "rope":
        T, n = c["T"], c["Hq"] + 2 * c["Hkv"]
        kept = c["Hq"] + 2 * c["Hkv"] * (1.0 - c["drop"])
        b = T * c["D"] * (n * (4 if c["dtype"] == "f32" else 2) + kept * 2) + 8 * T + 2 * c["rot"]
        return {"bytes": b + (8 * c["D"] if c["norm"] else 0), "flops": T * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + 4 * c["D"])}
    if c["op"] == "attention":
        S, shared, mine = _attention_rows(c)
        pairs = S * c["shared"] * (1.0 - c["ragged"] / 2) + mine
        if c["causal"]:   # query i of n sees shared - n + i + 1 keys
            pairs = S * (c["shared"] - (c["most"] - 1) / 2)
        b = 4 * (shared + mine) * c["Hkv"] * c["D"] + 4 * S * c["Hq"] * c["D"]
        return {"bytes": b + 4 * (shared + mine) / c["page"] + 8 * S, "flops": 4 * pairs * c["Hq"] * c["D"]}
    if c["op"] == "beam":
        n = c["groups"] * c["W"]
        return {"bytes": 4 * n * c["V"] + 5 * n + 13 * c["groups"] * c["K"], "flops": 4 * n * c["V"]}
    S = c["groups"] * c["W"]
    moved = S * (1.0 - 1.0 / c["W"])
    rows = (c["page"] - 1) / 2 if c["length"] >= 40 else min(c["length"], c["page"]) / 2
    return {"bytes": 2 * moved * c["planes"] * rows * c["Hkv"] * c["D"] * 2 + 8 * S * c["maxp"] + 16 * S, "flops": 0}


# ------------------------------------------------------------------------- the definition in 64 bits

def _exact_heads(x, gamma, angle, layout):
    """Each pair (a, b) of a head as the complex number a + ib, turned by its angle."""
    x = x.double().clone()
    if gamma is not None:
        x = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * gamma.double()
    half = angle.shape[1]
    at = torch.arange(half, device=DEV)
    a, b = (at, at + half) if layout == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_rows(cache, table, n, head):
    """Rows [0, n) of one kv head of a sequence, page by page of its table."""
    page = cache.shape[2]
    ids = table[: (n + page - 1) // page].long()
    return cache[ids, head].reshape(-1, cache.shape[3])[:n].double()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
        q = _exact_heads(s["q"], s["q_gamma"], angle, c["layout"])
        k = _exact_heads(s["k"], s["k_gamma"], angle, c["layout"])
        kc, vc = (s[n].double().permute(0, 2, 1, 3).flatten(0, 1) for n in ("k_cache", "v_cache"))
        live = s["slots"] >= 0
        kc[s["slots"][live].long()] = k[live]
        vc[s["slots"][live].long()] = s["v"][live].double()
        back = lambda m: m.reshape(-1, c["page"], c["Hkv"], c["D"]).permute(0, 2, 1, 3).contiguous()  # noqa: E731
        return [q, back(kc), back(vc)]
    if c["op"] == "attention":
        S, Hq, D = s["q"].shape
        G = Hq // c["Hkv"]
        first, shared = s["group_offsets"].tolist(), s["shared_lens"].tolist()
        own_lens = s["own_lens"].tolist() if s["own_lens"] is not None else [0] * S
        out = torch.zeros(S, Hq, D, device=DEV, dtype=torch.float64)
        for h in range(c["Hkv"]):
            for g in range(c["groups"]):
                a, b = first[g], first[g + 1]
                q = s["q"][a:b, h * G:(h + 1) * G].double()
                k = _exact_rows(s["k_cache"], s["shared_pages"][g], shared[g], h)
                v = _exact_rows(s["v_cache"], s["shared_pages"][g], shared[g], h)
                z = torch.exp(torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(D))
                if s["limits"] is not None:
                    z *= (torch.arange(shared[g], device=DEV)[None, :] < s["limits"][a:b, None])[:, None, :]
                den, num = z.sum(2), torch.einsum("tgk,kd->tgd", z, v)
                if s["own_lens"] is not None:
                    # the own segments of the group, one after another in one matrix; a row sees its own part
                    n = own_lens[a:b]
                    k, v = (torch.cat([_exact_rows(s[m], s["own_pages"][a + i], n[i], h) for i in range(b - a)])
                            for m in ("k_cache", "v_cache"))
                    if k.shape[0] > 0:
                        of = torch.repeat_interleave(torch.arange(b - a, device=DEV), torch.tensor(n, device=DEV))
                        z = torch.exp((q[of] * k[:, None, :]).sum(2) / math.sqrt(D))   # [keys][G]
                        den = den.index_add(0, of, z)
                        num = num.index_add(0, of, z[..., None] * v[:, None, :])
                out[a:b, h * G:(h + 1) * G] = torch.where(den[..., None] > 0, num / den[..., None], 0.0)
        return out
    if c["op"] == "beam":
        groups, W, K = c["groups"], c["W"], c["K"]
        best = torch.full((groups, K), float("-inf"), dtype=torch.float64)
        for g in range(groups):
            found = []
            for w in range(W):
                cum = float(s["scores"][g, w])
                if s["finished"][g, w]:
                    found.append(torch.tensor([cum], dtype=torch.float64))
                    continue
                p = torch.softmax(s["logits"][g * W + w].cpu().double(), 0)
                top = torch.topk(p, min(K, c["V"])).values
                found.append(cum + torch.log(top[top > 0]))
            top = torch.sort(torch.cat(found), descending=True).values[:K]
            best[g, :top.numel()] = top
        return [None, None, best, None]
    return None
