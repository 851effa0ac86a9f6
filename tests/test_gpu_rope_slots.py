"""Tokens that name the same slot of the cache."""
import pytest
from gpu_util import torch_cuda

import gemm_decode_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rot", [(128, 128), (64, 0), (17, 16)])
def test_a_shared_slot_holds_elements_of_its_tokens(D, rot):
    """Every element is one of the tokens' own, and no other row is touched."""
    torch = torch_cuda()
    torch.manual_seed(D)
    T, Hq, Hkv, page = 64, 4, 2, 16
    x = torch.randn(T, Hq + 2 * Hkv, D, device="cuda")
    positions = torch.arange(T, device="cuda", dtype=torch.int32)
    f = q4.q4_rope_frequencies(rot).cuda()

    def run(slots):
        pools = [torch.full((6, Hkv, page, D), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        out = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16)
        q4.q4_rope_append_run(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], positions, f, out, *pools, slots=slots)
        return [p.transpose(1, 2).reshape(6 * page, Hkv, D) for p in pools]

    apart = run(torch.arange(T, device="cuda", dtype=torch.int32))
    slots = (64 + torch.arange(T, device="cuda") % 3).to(torch.int32)
    for own, shared in zip(apart, run(slots)):
        for s in range(3):
            mine = own[:T][slots == 64 + s]
            assert (shared[64 + s][None] == mine).any(0).all()
        assert (shared[:64] == 7).all() and (shared[67:] == 7).all()
