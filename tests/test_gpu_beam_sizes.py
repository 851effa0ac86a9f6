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


def test_logits_whose_scores_round_alike(torch):
    """Within a beam the order is that of the logits, then the tokens, where binary64 scores are
    equal: logits far below the score's last bit, and beams' scores that swallow them."""
    V = 6000
    logits = torch.full((1, V), -20.0, device="cuda")
    at = [4100, 17, 5999, 2500]
    for i, v in enumerate(at):
        logits[0, v] = (i + 1) * 1e-17          # binary64 keeps 1e-16 of a score of some units
    logits[0, 40], logits[0, 30] = 4e-17, 2e-17   # as large as the last and the second
    zero = torch.zeros(1, 1, device="cuda")
    got = step(torch, logits, zero, 6)
    assert float(logits[0, 40]) == float(logits[0, 2500]) and float(logits[0, 30]) == float(logits[0, 17])
    assert got[0].tolist() == [[40, 2500, 5999, 17 if 17 < 30 else 30, 30, 4100]]
    assert step(torch, logits, zero, 2)[0].tolist() == [[40, 2500]]
    # two beams so far down that no logit moves their scores: the lower beam's logits in order
    logits = torch.randn(2, V, device="cuda")
    want = torch.sort(logits[0].double().cpu(), descending=True, stable=True).indices[:5].tolist()
    got = step(torch, logits, torch.full((1, 2), -1e30, device="cuda"), 5)
    assert got[0].tolist() == [want] and got[1].tolist() == [[0] * 5]
    # a finished beam beside a live one whose best continuation scores nearly the same
    logits = torch.full((2, V), -60.0, device="cuda")
    logits[1, 9] = 0.0                           # that beam's sum is 1 + 5999 e^-60: its best scores its own score
    done = torch.tensor([[1, 0]], device="cuda", dtype=torch.uint8)
    for first, parent in ((-1.0, 0), (-1.0 - 2.0 ** -20, 1)):
        got = step(torch, logits, torch.tensor([[first, -1.0]], device="cuda"), 2, finished=done, eos=3)
        assert got[1].tolist() == [[parent, 1 - parent]]
        assert got[0].tolist() == [[3, 9] if parent == 0 else [9, 3]] and got[3].tolist() == [[1, 0] if parent == 0 else [0, 1]]
