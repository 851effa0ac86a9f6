"""Rows, pages and planes that lie more than 2^32 elements apart, and the longest rows of logits."""
import decode_reference as ref
import pytest
from gpu_util import torch_cuda
from test_gpu_beam import step

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_cuda()
    yield t
    t.cuda.empty_cache()


def test_rotary_rows_and_pages_far_apart(torch):
    T, Hq, Hkv, D, page, far = 3, 4, 2, 64, 16, 2 ** 31
    rows = torch.empty(2 * far + 4096, device="cuda", dtype=torch.bfloat16)
    x = rows.as_strided((T, Hq + 2 * Hkv, D), (far, D, 1))
    x.copy_(torch.randn(T, Hq + 2 * Hkv, D, device="cuda"))
    pool = torch.empty(2 * far + 2 ** 20, device="cuda", dtype=torch.bfloat16)
    kc, vc = (pool[at:].as_strided((3, Hkv, page, D), (far, page * D, D, 1)) for at in (0, 2 ** 16))
    kc.fill_(7.0), vc.fill_(7.0)
    slots = torch.tensor([2 * page + 15, 3, page], device="cuda", dtype=torch.int32)
    positions = torch.tensor([5, 70000, 9], device="cuda", dtype=torch.int32)
    f = q4.q4_rope_frequencies(D)
    out = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16)
    q4.q4_rope_append_run(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], positions, f.cuda(), out, kc, vc, slots=slots)
    for got, part in ((out, x[:, :Hq]), (torch.stack([kc[int(s) // page, :, int(s) % page] for s in slots]), x[:, Hq:Hq + Hkv])):
        want, bound = ref.rope(part, None, positions, f, True, 1.0, 1e-6)
        ref.within(got, want, (1 + 2.0 ** -7) * bound + ref.rounding(want, torch.bfloat16), "rotated")
    assert torch.equal(torch.stack([vc[int(s) // page, :, int(s) % page] for s in slots]), x[:, Hq + Hkv:])
    assert int((kc == 7).all(3).sum()) == (3 * page - T) * Hkv


def test_pages_of_a_reordering_far_apart(torch):
    planes, heads, page, D, far = 2, 2, 16, 32, 2 ** 31
    flat = torch.empty(3 * far + 2 ** 20, device="cuda", dtype=torch.bfloat16)
    pool = flat.as_strided((planes, 4, heads, page, D), (4096, far, page * D, D, 1))
    pool.copy_(torch.randint(-90, 90, pool.shape, device="cuda"))
    i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    tables, spare, lens, parents = i32([0], [3]), i32(2, 1), i32(11), i32([1, 0])
    new, left = torch.empty_like(tables), torch.empty_like(spare)
    want = ref.reorder(tables.cpu(), lens.cpu(), parents.cpu(), spare.cpu(), pool.cpu())
    q4.q4_beam_reorder_run(tables, lens, parents, spare, new, left, pool)
    assert torch.equal(new.cpu(), want[0]) and torch.equal(left.cpu(), want[1]) and torch.equal(pool.cpu(), want[2])


def test_logits_far_apart(torch):
    rows, V, stride = 36, 5000, 2 ** 27
    flat = torch.empty((rows - 1) * stride + V, device="cuda")
    logits = flat.as_strided((rows, V), (stride, 1))
    logits.copy_(3 * torch.randn(rows, V, device="cuda"))
    scores = -9 * torch.rand(3, 12, device="cuda")
    near = step(torch, logits.contiguous(), scores, 8)
    assert all(torch.equal(a, b) for a, b in zip(step(torch, logits, scores, 8), near))
    want = ref.beam_step(logits.cpu(), scores.cpu(), None, 8, -1)
    assert torch.equal(near[0].cpu().long(), want[0]) and torch.equal(near[1].cpu().long(), want[1])


def test_the_longest_row_of_logits(torch):
    """2^31 - 2 logits, the best in the last chunk, the first and at the borders of the parts."""
    V = 2 ** 31 - 2
    logits = torch.full((1, V), -40.0, device="cuda")
    at = [V - 1, 0, 2 ** 30, 65536, V - 70000, 65535, 4096, 2 ** 25]
    for i, v in enumerate(at):
        logits[0, v] = 9.0 - i
    tokens, parents, scores, _ = step(torch, logits, torch.zeros(1, 1, device="cuda"), 9)
    first = min(set(range(9)) - set(at))   # (the ninth: the lowest token of all others)
    assert tokens.tolist() == [at + [first]] and parents.tolist() == [[0] * 9]
    # the sum: eight large terms and 2^31 of e^-49 of the largest (1e-12 of it in all)
    want = torch.log_softmax(torch.tensor([9.0 - i for i in range(8)], dtype=torch.float64), 0)
    assert (scores[0, :8].cpu().double() - want).abs().max() <= 2.0 ** -21 + 40 * 2.0 ** -24 + 2.0 ** -24 * 8
