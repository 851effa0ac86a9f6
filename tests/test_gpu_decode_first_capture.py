"""The calls for several continuations of one prompt, captured into a graph by a process that has
made no call before: nothing that a first call looks up may be refused during a capture."""
import os
import subprocess
import sys

import pytest
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import torch
import gemm_decode_gb300 as q4

T, Hq, Hkv, D, page, V, W, K = 24, 8, 2, 128, 16, 9000, 12, 8
i32 = dict(device="cuda", dtype=torch.int32)
bf = dict(device="cuda", dtype=torch.bfloat16)
torch.manual_seed(0)
x = torch.randn(T, Hq + 2 * Hkv, D, device="cuda")
pool = torch.randn(2, 40 + 2 * T, Hkv, page, D, device="cuda").to(torch.bfloat16)
f = torch.rand(D // 2, device="cuda")
positions = torch.arange(T, **i32)
shared = torch.arange(40, **i32)[None]
own = torch.arange(40, 40 + T, **i32)[:, None].contiguous()
spare, slots = own[:, 0] + T, own[:, 0] * page
logits, scores = torch.randn(T, V, device="cuda"), -torch.rand(T // W, W, device="cuda")
n, one, lens = torch.full((1,), 600, **i32), torch.ones(T, **i32), torch.ones(T // W, **i32)
# (no call before the capture, so its size is looked at below)
work = torch.empty(1 << 26, device="cuda", dtype=torch.uint8)


def outputs():
    return dict(q=torch.zeros(T, Hq, D, **bf), o=torch.zeros(T, Hq, D, **bf), tokens=torch.zeros(T // W, K, **i32),
                parents=torch.zeros(T // W, K, **i32), best=torch.zeros(T // W, K, device="cuda"),
                tables=torch.zeros_like(own), left=torch.zeros_like(spare), pool=pool.clone())


def step(r):
    k, v = r["pool"][0], r["pool"][1]
    q4.q4_rope_append_run(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], positions, f, r["q"], k, v, slots=slots)
    q4.q4_prefix_attn_run(r["q"], k, v, r["o"], work, shared_pages=shared, shared_lens=n, own_pages=own, own_lens=one,
                          flags=q4.Q4_RUN_OVERLAPPED)
    q4.q4_beam_step_run(logits, scores, r["tokens"], r["parents"], r["best"], work)
    back = (torch.arange(T // W * W, **i32).view(T // W, W) * 5 + 1) % W
    q4.q4_beam_reorder_run(own, lens, back.to(torch.int32), spare, r["tables"], r["left"], r["pool"])


first = outputs()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step(first)
graph.replay()
torch.cuda.synchronize()
again = outputs()
step(again)
torch.cuda.synchronize()
assert work.numel() >= max(q4.q4_prefix_attn_workspace(T, 1, Hq, Hkv, D), q4.q4_beam_step_workspace(T // W, W, K, V))
assert q4.q4gemv_device_status() == q4.Q4_OK
for name in first:
    assert torch.equal(first[name], again[name]), name
assert torch.isfinite(first["o"]).all() and (first["o"] != 0).any()
print("captured")
"""


def test_a_first_call_may_be_captured():
    torch_cuda()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
