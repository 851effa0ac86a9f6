"""Beam steps of sizes where the work is divided in other ways: more rows than 2^16, and chunks of
more logits than a CTA holds the maxima of at a time."""
import pytest
from gpu_util import torch_cuda
from test_gpu_beam import step

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def by_definition(torch, logits, scores, K):
    """(tokens, parents, scores) in binary64, a group at a time sorted as a whole, on the GPU."""
    groups, W = scores.shape
    V = logits.shape[1]
    s = torch.log_softmax(logits.double(), 1).view(groups, W * V) + scores.double().repeat_interleave(V, 1)
    s, at = (t[:, :K] for t in torch.sort(s, dim=1, descending=True, stable=True))
    return at % V, at // V, s


def same(torch, got, want, V):
    """Equal choices: these inputs have no two beams whose scores are closer than the sums of
    exponentials are known (test_gpu_beam.check: 2^-21 and V / 4096 + 24 steps)."""
    lost = 2.0 ** -21 + (V / 4096 + 24) * 2.0 ** -24
    assert ((got[2].double() - want[2]).abs() <= lost + 2.0 ** -24 * want[2].abs()).all()
    wrong = (got[0] != want[0]) | (got[1] != want[1])
    if not wrong.any():
        return
    for g in torch.nonzero(wrong.any(1))[:, 0].tolist():   # then only neighbours as close as that
        first = {(int(v), int(w)): float(x) for v, w, x in zip(want[0][g], want[1][g], want[2][g])}
        for j in torch.nonzero(wrong[g])[:, 0].tolist():
            at = (int(got[0][g, j]), int(got[1][g, j]))
            assert at in first and abs(first[at] - float(want[2][g, j])) <= 2 * lost, (g, j)


@pytest.mark.parametrize("groups,W,K,V", [(16400, 4, 3, 5), (70000, 1, 2, 3), (2100, 32, 4, 2)])
def test_more_rows_than_65535(torch, groups, W, K, V):
    torch.manual_seed(groups)
    logits = 3 * torch.randn(groups * W, V, device="cuda")
    scores = -9 * torch.rand(groups, W, device="cuda")
    same(torch, step(torch, logits, scores, K), by_definition(torch, logits, scores, K), V)


@pytest.mark.parametrize("rows,W,K,V", [(620, 10, 8, 70001), (608, 16, 32, 65537), (640, 16, 4, 140000)])
def test_chunks_of_several_parts(torch, rows, W, K, V):
    """As many rows as CTAs: a row is one chunk, whose maxima are held 65536 logits at a time."""
    torch.manual_seed(V)
    logits = 3 * torch.randn(rows, V, device="cuda")
    logits[1] = torch.linspace(-4, 4, V, device="cuda")             # the best in the last part
    logits[2] = torch.linspace(4, -4, V, device="cuda")             # and in the first
    logits[3] = 0.0                                                 # all the same: the first tokens
    logits[4, 65536:] = float("-inf")
    logits[5, :65536] = float("-inf")
    logits[6, 65530:65540] = 30.0                                   # across the border
    scores = -9 * torch.rand(rows // W, W, device="cuda")
    scores[0] = -torch.arange(W, device="cuda") * 0.01
    part = [slice(g, g + 8) for g in range(0, rows // W, 8)]
    got = step(torch, logits, scores, K)
    for p in part:
        want = by_definition(torch, logits[p.start * W:p.stop * W], scores[p], K)
        same(torch, [t[p] for t in got[:3]], want, V)


def test_chunks_follow_the_device(torch):
    """One row is split into as many chunks as there are blocks of 4096 logits, up to 64, and many
    rows into so many that four CTAs an SM have one each; a chunk leaves K keys and two sums."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for rows, K, V in ((1, 4, 4097), (1, 1, 10 ** 6), (64, 8, 128256), (sms, 2, 50000), (4 * sms, 3, 50000), (5 * sms, 1, 9000)):
        blocks = -(-V // 4096)
        want = min(blocks, max(4 * sms // rows, 1), 64)
        chunk = -(-(-(-V // want)) // 32) * 32
        bytes_ = rows * -(-V // chunk) * (8 + 8 * K)
        assert q4.q4_beam_step_workspace(rows, 1, K, V) == -(-bytes_ // 256) * 256 + 256
