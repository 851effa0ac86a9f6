#!/usr/bin/env python3
"""A mixture-of-experts feed-forward block over int4 experts, as a model's layer keeps it.

`MoeBlock` holds the weights, the workspace and the outputs of one layer, and runs the
router, the experts and the norms that follow as one call.  The router's logits come from the
model: for up to 16 tokens from the library's dense GEMV, for prompts from any matrix product.

    python examples/moe_block.py            # checks a layer against a plain one and times it
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gemm_decode_gb300 as q4  # noqa: E402


class MoeBlock:
    """One layer: x' = residual_scale x + gate norm(sum of the experts), and norm(x')."""

    def __init__(self, up, down, router, post_gamma, pre_gamma, gate, top_k, group, most_tokens, dtype,
                 score=q4.Q4_ROUTE_SOFTMAX, residual_scale=1.0, eps=1e-6):
        import torch
        self.up, self.down, self.router = up, down, router          # router: float32 [experts, hidden]
        self.norms = dict(post_gamma=post_gamma, pre_gamma=pre_gamma, gate=gate, residual_scale=residual_scale, eps=eps)
        self.top_k, self.group, self.score, self.most = top_k, group, score, most_tokens
        experts, hidden, inner = up[0].shape[0], down[0].shape[1], 2 * down[0].shape[2]
        dev = up[0].device
        n = q4.q4moe_block_workspace(most_tokens, experts, top_k, hidden, inner, dtype)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        self.ids = torch.empty(most_tokens, top_k, dtype=torch.int32, device=dev)
        self.weights = torch.empty(most_tokens, top_k, device=dev)

    def logits(self, a):
        """Router logits of the normed input, [tokens, experts]."""
        import torch
        if a.shape[0] > 16:
            return a.float() @ self.router.T
        out = torch.empty(a.shape[0], self.router.shape[0], device=a.device)
        q4.f32gemv_run(self.router, a.float(), out)
        return out

    def __call__(self, a, x, out=None, normed=None):
        """a: the normed input, x: the residual stream, [tokens, hidden]; returns the new
        stream and its norm, the next block's input."""
        import torch
        T = x.shape[0]
        if T > self.most:
            raise ValueError(f"{T} tokens: the workspace was made for {self.most}")
        out = torch.empty_like(x) if out is None else out
        normed = torch.empty_like(x) if normed is None else normed
        q4.q4moe_block_run(self.up, self.down, self.logits(a), a, x, out, normed, self.ids[:T], self.weights[:T],
                           self.workspace, group=self.group, score=self.score, **self.norms)
        return out, normed


def random_experts(experts, rows, cols, group, generator):
    """Random int4 experts in the MatMulNBits layout: codes, scales, zero points."""
    import torch
    dev = generator.device
    codes = torch.randint(0, 256, (experts, rows, cols // 2), dtype=torch.uint8, device=dev, generator=generator)
    scales = (0.002 + 0.006 * torch.rand(experts, rows, cols // group, device=dev, generator=generator)).half()
    zeros = torch.randint(0, 256, (experts, rows, (cols // group + 1) // 2), dtype=torch.uint8, device=dev,
                          generator=generator)
    return codes, scales, zeros


def random_block(dtype, hidden, inner, experts, top_k, group, most_tokens, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    up = random_experts(experts, 2 * inner, hidden, group, g)
    down = random_experts(experts, hidden, inner, group, g)
    router = torch.randn(experts, hidden, device="cuda", generator=g) / hidden ** 0.5
    post, pre = (0.5 + torch.rand(hidden, device="cuda", generator=g) for _ in range(2))
    gate = (1.0 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).to(dtype)
    return MoeBlock(up, down, router, post, pre, gate, top_k, group, most_tokens, dtype)


def plain(block, a, x):
    """The block in 64 bits, token by token."""
    import torch

    def matrix(w, e):
        codes, scales, zeros = (t[e].cpu() for t in w)
        q = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).double()
        z = torch.stack([zeros & 15, zeros >> 4], -1).reshape(zeros.shape[0], -1)[:, :scales.shape[1]].double()
        grow = lambda t: t.double().repeat_interleave(block.group, 1)  # noqa: E731
        return (q - grow(z)) * grow(scales)

    logits = block.logits(a).cpu().double()
    out = []
    for t in range(x.shape[0]):
        chosen = torch.sort(logits[t], descending=True, stable=True).indices[:block.top_k]
        w = torch.softmax(logits[t][chosen], 0)
        b = torch.zeros(x.shape[1], dtype=torch.float64)
        for e, p in zip(chosen.tolist(), w):
            v = matrix(block.up, e) @ a[t].cpu().double()
            b += p * (matrix(block.down, e) @ (torch.nn.functional.silu(v[0::2]) * v[1::2]))
        n = block.norms
        rms = lambda v, gamma: v / torch.sqrt((v * v).mean() + n["eps"]) * gamma.cpu().double()  # noqa: E731
        new = n["residual_scale"] * x[t].cpu().double() + n["gate"].cpu().double() * rms(b, n["post_gamma"])
        out.append(torch.stack([new, rms(new, n["pre_gamma"])]))
    return torch.stack(out, 1)


def check(dtype, hidden, inner, experts, top_k, group):
    """Largest relative error (2-norm) of a prompt of 40 tokens and of single tokens replayed
    from a CUDA graph, against the plain block."""
    import torch
    block = random_block(dtype, hidden, inner, experts, top_k, group, 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    worst = 0.0

    def compare(a, x, got):
        want = plain(block, a, x)
        for have, w in zip(got, want):
            worst_now = float((have.cpu().double() - w).norm() / w.norm())
            nonlocal worst
            worst = max(worst, worst_now)

    a, x = (torch.randn(40, hidden, device="cuda", generator=g).to(dtype) for _ in range(2))
    compare(a, x, block(a, x))
    a, x = a[:1].clone(), x[:1].clone()
    out, normed = torch.empty_like(x), torch.empty_like(x)
    block(a, x, out, normed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(a, x, out, normed)
    for _ in range(3):
        a.copy_(torch.randn(1, hidden, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        compare(a, x, (out, normed))
    return worst


def main():
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        print(f"{dtype}: relative error {check(dtype, 512, 256, 8, 2, 64):.2g}")
    block = random_block(torch.bfloat16, 2048, 1024, 64, 8, 128, 2048)
    for tokens in (1, 8, 64, 2048):
        a, x = (torch.randn(tokens, 2048, device="cuda").bfloat16() for _ in range(2))
        out, normed = torch.empty_like(x), torch.empty_like(x)
        for _ in range(3):
            block(a, x, out, normed)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        for _ in range(20):
            block(a, x, out, normed)
        end.record()
        torch.cuda.synchronize()
        print(f"{tokens} tokens, 64 experts of 2048 x 1024, 8 per token: {start.elapsed_time(end) * 50:.1f} us")


if __name__ == "__main__":
    main()
