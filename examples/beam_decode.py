#!/usr/bin/env python3
"""Beam search over a small int4 transformer: the attention side of its layers, the LM head and
the search as a program keeps them.

A group of beams shares its prompt's keys and values, which the prompt's pass puts into the
paged cache once; each beam has pages of its own for what it continues with.  A step is the
decode GEMVs, the rotary call, the attention over the shared and the own pages, the LM head,
the choice of continuations, and the reordering of pages.  Nothing of it needs the host: the
step is captured in a CUDA graph once and replayed.

    python examples/beam_decode.py          # checks a search against a plain one and times a step
"""
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gemm_decode_gb300 as q4  # noqa: E402


class Matrix:
    """An int4 matrix of group 32, y = W x: up to 16 rows of x as GEMVs, more as a matmul."""

    def __init__(self, rows, cols, scale, generator):
        import torch
        dev = generator.device
        self.codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device=dev, generator=generator)
        self.scales = (scale * (0.5 + torch.rand(rows, cols // 32, device=dev, generator=generator))).half()

    def gemv(self, x, y, gamma=None, eps=1e-6):
        """With gamma, of x's norm.  At most 16 rows a call."""
        for i in range(0, x.shape[0], 16):
            part, to = x[i:i + 16], y[i:i + 16]
            if gamma is None:
                q4.q4gemv_run(self.codes, self.scales, None, part, to)
            else:
                q4.q4gemv_fused_run(self.codes, self.scales, None, part, gamma, eps, to)
        return y

    def gemm(self, a):
        import torch
        c = torch.empty(a.shape[0], self.codes.shape[0], device=a.device)
        q4.q4gemm_run(self.codes, self.scales, None, a, c)
        return c

    def plain(self):
        import torch
        q = torch.stack([self.codes & 15, self.codes >> 4], -1).flatten(1).double().cpu()
        return (q - 8) * self.scales.double().cpu().repeat_interleave(32, 1)


class Model:
    def __init__(self, layers, hidden, Hq, Hkv, D, vocabulary, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.Hq, self.Hkv, self.D, self.V = hidden, Hq, Hkv, D, vocabulary
        rand = lambda *n: torch.randn(*n, device="cuda", generator=g)  # noqa: E731
        self.embedding = rand(vocabulary, hidden)
        near1 = lambda n: 1.0 + 0.1 * rand(n)  # noqa: E731
        unit = 0.2 / math.sqrt(hidden)   # codes are 4.6 on average
        self.layers = [dict(norm=near1(hidden), q_gamma=near1(D), k_gamma=near1(D),
                            qkv=Matrix((Hq + 2 * Hkv) * D, hidden, unit, g),
                            out=Matrix(hidden, Hq * D, 0.2 / math.sqrt(Hq * D), g)) for _ in range(layers)]
        self.norm, self.head = near1(hidden), Matrix(vocabulary, hidden, unit, g)
        self.inv_freq = q4.q4_rope_frequencies(D, 10000.0).cuda()


class Beams:
    """`width` beams for each of some prompts, of at most `most` further tokens."""

    def __init__(self, model, prompts, width, most, eos, page=16):
        import torch
        m, i32, dev = model, torch.int32, "cuda"
        self.model, self.W, self.page, self.eos = model, width, page, eos
        self.groups = len(prompts)
        S = self.S = self.groups * width
        need = [(len(p) + page - 1) // page for p in prompts]
        self.columns = (most + page - 1) // page + 1
        pages = sum(need) + S * (self.columns + 1)
        self.pool = torch.zeros(2 * len(m.layers), pages, m.Hkv, page, m.D, device=dev, dtype=torch.bfloat16)
        # the prompts' pages, then a column of pages for each beam written ahead, then a spare one each
        self.shared_pages = torch.zeros(self.groups, max(need), dtype=i32, device=dev)
        at = 0
        for g, n in enumerate(need):
            self.shared_pages[g, :n] = torch.arange(at, at + n)
            at += n
        self.tables = (at + torch.arange(S * self.columns)).reshape(S, self.columns).to(dev, i32)
        self.spare = (at + S * self.columns + torch.arange(S)).to(dev, i32)
        self.shared_lens = torch.tensor([len(p) for p in prompts], dtype=i32, device=dev)
        self.group_offsets = (torch.arange(self.groups + 1) * width).to(dev, i32)
        self.lens = torch.zeros(self.groups, dtype=i32, device=dev)
        self.scores = torch.zeros(self.groups, width, device=dev)
        self.finished = torch.zeros(self.groups, width, dtype=torch.uint8, device=dev)
        self.tokens, self.parents = (torch.zeros(self.groups, width, dtype=i32, device=dev) for _ in range(2))
        self.logits = torch.empty(S, m.V, device=dev)
        self.new = dict(tables=torch.empty_like(self.tables), spare=torch.empty_like(self.spare),
                        tokens=torch.empty_like(self.tokens), parents=torch.empty_like(self.parents),
                        scores=torch.empty_like(self.scores), finished=torch.empty_like(self.finished))
        bytes_ = max(q4.q4_prefix_attn_workspace(max(S, sum(map(len, prompts))), self.groups, m.Hq, m.Hkv, m.D),
                     q4.q4_beam_step_workspace(self.groups, width, width, m.V))
        self.workspace = torch.empty(bytes_, dtype=torch.uint8, device=dev)
        self._prompt(prompts)

    def _attend(self, layer, qkv, positions, slots, out, **segments):
        """The layer's rotary call and attention over a product's rows [tokens, (Hq + 2 Hkv) D]."""
        import torch
        m, w = self.model, self.model.layers[layer]
        heads = qkv.unflatten(1, (-1, m.D))
        q = torch.empty(qkv.shape[0], m.Hq, m.D, device=qkv.device, dtype=self.pool.dtype)
        keys, values = self.pool[2 * layer], self.pool[2 * layer + 1]
        q4.q4_rope_append_run(heads[:, :m.Hq], heads[:, m.Hq:m.Hq + m.Hkv], heads[:, m.Hq + m.Hkv:], positions,
                              m.inv_freq, q, keys, values, slots=slots, q_gamma=w["q_gamma"], k_gamma=w["k_gamma"])
        q4.q4_prefix_attn_run(q, keys, values, out, self.workspace, shared_pages=self.shared_pages,
                              shared_lens=self.shared_lens, **segments)
        return out

    def _choose(self):
        """Continuations from the logits, and the pages that follow them."""
        n = self.new
        q4.q4_beam_step_run(self.logits, self.scores, n["tokens"], n["parents"], n["scores"], self.workspace,
                            finished=self.finished, out_finished=n["finished"], eos=self.eos)
        q4.q4_beam_reorder_run(self.tables, self.lens, n["parents"], self.spare, n["tables"], n["spare"], self.pool)
        for name, value in n.items():
            getattr(self, name).copy_(value)

    def _prompt(self, prompts):
        import torch
        m, i32 = self.model, torch.int32
        lens = [len(p) for p in prompts]
        flat = torch.tensor([t for p in prompts for t in p], device="cuda")
        positions = torch.cat([torch.arange(n) for n in lens]).to("cuda", i32)
        of = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
        slots = (self.shared_pages[of, positions.long() // self.page] * self.page + positions % self.page).to(i32)
        offsets = torch.tensor([sum(lens[:g]) for g in range(len(lens) + 1)], dtype=i32, device="cuda")
        x = m.embedding[flat]
        for layer, w in enumerate(m.layers):
            a = (x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * w["norm"]).bfloat16()
            out = torch.empty(len(flat), m.Hq, m.D, device="cuda", dtype=torch.bfloat16)
            self._attend(layer, w["qkv"].gemm(a), positions, slots, out, group_offsets=offsets, limits=positions + 1)
            x = x + w["out"].gemm(out.flatten(1))
        last = x[offsets[1:].long() - 1].contiguous()
        first = m.head.gemv(last, torch.empty(self.groups, m.V, device="cuda"), m.norm)
        self.logits.copy_(first.repeat_interleave(self.W, 0))
        self.scores.fill_(-math.inf)   # all beams are the same so far: the first alone goes on
        self.scores[:, 0] = 0.0
        self._choose()

    def step(self):
        """One token for every beam."""
        import torch
        m, i32 = self.model, torch.int32
        n = self.lens.repeat_interleave(self.W)
        positions = self.shared_lens.repeat_interleave(self.W) + n
        slots = torch.gather(self.tables, 1, (n // self.page).long()[:, None])[:, 0] * self.page + n % self.page
        x = m.embedding[self.tokens.flatten().long().clamp_min(0)]
        for layer, w in enumerate(m.layers):
            qkv = w["qkv"].gemv(x, torch.empty(self.S, (m.Hq + 2 * m.Hkv) * m.D, device=x.device), w["norm"])
            out = torch.empty(self.S, m.Hq, m.D, device=x.device)
            self._attend(layer, qkv, positions.to(i32), slots.to(i32), out, group_offsets=self.group_offsets,
                         own_pages=self.tables, own_lens=(n + 1).to(i32))
            x = x + w["out"].gemv(out.flatten(1), torch.empty_like(x))
        m.head.gemv(x, self.logits, m.norm)
        self.lens += 1
        self._choose()


def plain_logits(model, prompt, continued):
    """Logits of the last token of a text in 64 bits, with the roundings of the path it takes:
    the prompt's products have bfloat16 operands, queries, keys and values are bfloat16."""
    import torch
    m, n = model, len(prompt)
    bf = lambda v: v.bfloat16().double()  # noqa: E731
    rms = lambda v, gamma: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * gamma.double().cpu()  # noqa: E731
    x = m.embedding.cpu().double()[torch.tensor(prompt + continued)]
    T = x.shape[0]
    angle = torch.arange(T).double()[:, None] * m.inv_freq.double().cpu()
    c, s = angle.cos()[:, None], angle.sin()[:, None]

    def turned(v):
        a, b = v.chunk(2, -1)
        return torch.cat([a * c - b * s, s * a + c * b], -1)

    for w in m.layers:
        a, wq = rms(x, w["norm"]), w["qkv"].plain()
        qkv = torch.cat([bf(a[:n]) @ bf(wq).T, a[n:] @ wq.T]).unflatten(1, (-1, m.D))
        q = bf(turned(rms(qkv[:, :m.Hq], w["q_gamma"])))
        k = bf(turned(rms(qkv[:, m.Hq:m.Hq + m.Hkv], w["k_gamma"]))).repeat_interleave(m.Hq // m.Hkv, 1)
        v = bf(qkv[:, m.Hq + m.Hkv:]).repeat_interleave(m.Hq // m.Hkv, 1)
        z = torch.einsum("thd,shd->hts", q, k) / math.sqrt(m.D)
        z = z.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
        o = torch.einsum("hts,shd->thd", torch.softmax(z, -1), v).flatten(1)
        wo = w["out"].plain()
        x = x + torch.cat([bf(o[:n]) @ bf(wo).T, o[n:] @ wo.T])
    return rms(x[-1], m.norm) @ m.head.plain().T


def check(prompts, width, steps, layers=2, hidden=256, Hq=4, Hkv=2, D=64, vocabulary=500):
    """Runs a search, its step replayed from a graph, and compares each beam's logits with a plain
    pass over its text.  Returns the largest relative error (2-norm) and, for each step, what the
    choice was made from and what it was: (logits, scores, finished, tokens, parents)."""
    import torch
    model = Model(layers, hidden, Hq, Hkv, D, vocabulary)
    beams = Beams(model, prompts, width, steps + 2, eos=7)
    texts = [[[int(t)] for t in row] for row in beams.tokens.cpu()]
    # a step outside the graph first (it sets the kernels up), then the graph
    worst, record, graph = 0.0, [], None
    for i in range(steps):
        before = beams.scores.clone(), beams.finished.clone()
        if i == 0:
            beams.step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    beams.step()
            graph.replay()
        torch.cuda.synchronize()
        logits = beams.logits.cpu().double()
        for g, prompt in enumerate(prompts):
            for w in range(width):
                if not before[1][g, w]:
                    want = plain_logits(model, prompt, texts[g][w])
                    worst = max(worst, float((logits[g * width + w] - want).norm() / want.norm()))
        record.append((beams.logits.clone(), *before, beams.tokens.clone(), beams.parents.clone()))
        texts = [[texts[g][int(beams.parents[g, w])] + [int(beams.tokens[g, w])] for w in range(width)]
                 for g in range(len(prompts))]
    return worst, record


def main():
    import torch
    worst, _ = check([list(range(40, 77)), [3, 1, 4, 1, 5], list(range(100, 164))], 4, 20)
    print(f"relative error of the logits against a plain pass: {worst:.2g}")
    model = Model(2, 4096, 32, 8, 128, 32000)
    prompts = [torch.randint(0, 32000, (n,)).tolist() for n in (4000, 2500)]
    beams = Beams(model, prompts, 4, 256, eos=2)
    beams.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beams.step()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"2 prompts, 4 beams each, 2 layers of 32 + 2 x 8 heads, 32000 tokens: {start.elapsed_time(end) * 10:.1f} us a step")


if __name__ == "__main__":
    main()
