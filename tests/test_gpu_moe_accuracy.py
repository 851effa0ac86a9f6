"""The accuracy of the expert products, within bounds of each kernel's own arithmetic
(moe_bounds.py; test_moe_bounds.py shows what these tell apart)."""
import moe_bounds as mb
import moe_reference as ref
import numpy as np
import pytest
from gpu_util import torch_cuda
from test_gpu_moe import groups, make_weights, num, run_experts, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return torch_cuda()


def products(torch, seed, E, k, T, N, K, g, sym, swiglu, bf16, x=None, zero_column=None):
    """(got, want, bound) of one call over random experts."""
    rng = np.random.default_rng(seed)
    weights = make_weights(rng, E, N, K, g, sym)
    if zero_column is not None:   # code 8 under the implied zero point: no weight
        byte = weights[0][..., zero_column // 2]
        weights[0][..., zero_column // 2] = byte & 0xF0 | 8 if zero_column % 2 == 0 else byte & 0x0F | 0x80
    offsets, rows = groups(rng, E, k, T, "even")
    x = rng.normal(0, 1, (T, K)) if x is None else x
    x = num(torch.from_numpy(x).to(torch.bfloat16 if bf16 else torch.float32))
    y = num(run_experts(torch, weights, g, x, rows, offsets, T * k, swiglu, bf16))
    want, bound = mb.experts(ref.dequant(*weights, g), x, rows, offsets, np.full(y.shape, 7.0), swiglu, bf16, g)
    return y, want, bound


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("E,k,T,N,K,g", [
    (1, 1, 1, 8, 32, 32), (4, 2, 5, 130, 96, 32), (6, 3, 40, 258, 832, 64), (3, 1, 100, 130, 896, 128),
    (5, 1, 700, 260, 320, 64), (2, 2, 150, 200, 1152, 128), (16, 2, 33, 64, 4864, 32), (2, 1, 90, 136, 4864, 128)])
def test_products_within_their_arithmetic(torch, bf16, swiglu, E, k, T, N, K, g):
    for sym in (False, True):
        got, want, bound = products(torch, K + T, E, k, T, N, K, g, sym, swiglu, bf16)
        within(got, want, bound, f"sym {sym}")


@pytest.mark.parametrize("T", [5, 20, 100])   # 16, 32 and 64 rows of x where the group allows them
@pytest.mark.parametrize("K,g", [(512, 32), (2048, 128), (2048, 64), (4864, 32), (4864, 128), (14336, 128)])
def test_binary32_products_in_the_2_norm(torch, T, K, g):
    got, want, bound = products(torch, K + T, 2, 2, T, 160, K, g, False, False, False)
    within(got, want, bound, "y")
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= mb.two_norm(K, g), off


@pytest.mark.parametrize("K,g", [(512, 32), (2048, 64), (4864, 128)])
def test_bfloat16_weights_are_exact_up_to_24_rows_per_expert(torch, K, g):
    """Nearly every output is the exact value's own rounding to bfloat16."""
    got, want, _ = products(torch, K, 2, 2, 20, 800, K, g, False, False, True)
    rounded = num(torch.from_numpy(want).to(torch.bfloat16))
    assert float((got != rounded).mean()) <= mb.MISROUNDED


@pytest.mark.parametrize("bf16,T,outlier", [(False, 5, 1e5), (False, 40, 1e9), (True, 5, 2.0 ** 20), (True, 5, 2.0 ** 34),
                                            (True, 150, 2.0 ** 20), (True, 150, 2.0 ** 34)])
def test_outliers_leave_the_others_what_is_stated(torch, bf16, T, outlier):
    """An element far above the rest of its row, without and with a weight: 2^-39 of it may be
    lost of each of the others."""
    rng = np.random.default_rng(T)
    x = rng.normal(0, 1, (T, 640))
    x[:, 77] = outlier
    got, want, bound = products(torch, T, 2, 1, T, 140, 640, 32, True, False, bf16, x=x, zero_column=77)
    within(got, want, bound, "no weight on the outlier")
    assert np.abs(want).max() < 100 * 640
    got, want, bound = products(torch, T, 2, 1, T, 140, 640, 32, True, False, bf16, x=x)
    within(got, want, bound, "a weight on the outlier")
    if bf16 and outlier < 2.0 ** 30 and T <= 48:   # above 2^-31 of the largest nothing is lost
        got, want, _ = products(torch, T, 2, 1, T, 140, 640, 32, True, False, bf16, x=x, zero_column=77)
        assert float((got != num(torch.from_numpy(want).to(torch.bfloat16))).mean()) <= 2 * mb.MISROUNDED
