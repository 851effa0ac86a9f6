"""The calls for several continuations of one prompt in a row, as a search uses them: prompts,
steps replayed from a graph, pages that fill up and change hands."""
import os
import sys

import decode_reference as ref
import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("lens,width,steps,heads", [((37, 5, 64), 4, 36, (4, 2, 64)), ((200,), 8, 20, (8, 1, 128)),
                                                    ((1, 16, 17, 15), 5, 18, (6, 2, 64)), ((90,), 1, 4, (2, 2, 64))])
def test_a_search_follows_a_plain_one(lens, width, steps, heads):
    torch = torch_cuda()
    import beam_decode
    assert q4.lib()._name == q4build.LIB_PATH
    torch.manual_seed(sum(lens))
    prompts = [torch.randint(0, 500, (n,)).tolist() for n in lens]
    worst, record = beam_decode.check(prompts, width, steps, Hq=heads[0], Hkv=heads[1], D=heads[2])
    # What the plain pass does not round as the path does: the weights of the values (bfloat16,
    # half a step 2^-8 of each), and what a value next to a rounding's border costs when it falls
    # to the other side (a step, 2^-7, of queries, keys or values, rarely).  In each of the two layers
    # that is 2^-8 of the attention's output at most, which is about as large as the stream it is
    # added to; a wrong key, position or page changes the output by its own size.
    assert worst <= 2 * 2 * 2.0 ** -8
    for logits, scores, finished, tokens, parents in record:
        want = ref.beam_step(logits.cpu(), scores.cpu(), finished.cpu(), width, 7)
        assert torch.equal(tokens.cpu().long(), want[0]) and torch.equal(parents.cpu().long(), want[1])
    assert q4.q4gemv_device_status() == q4.Q4_OK
