"""A bias of FP32's lowest value under groups: the sum of two such c is -inf, yet the experts can be chosen (the marker of
a disabled expert that is a value, as test_gpu_router_grouped.py has it for logits)."""
import numpy as np
import pytest
import torch

from oracle import router as R
from test_gpu_router_grouped import biases, check, logits

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_groups_whose_sum_leaves_fp32(score, renorm):
    z = torch.zeros(3, 8)
    b = torch.full((8,), LOW)
    b[:2] = 0
    f = check(z, 4, b, 4, 2, score, renorm)
    assert f["idx"].tolist() == [[0, 1, 2, 3]] * 3
    f = check(z, 4, torch.full((8,), LOW), 4, 2, score, renorm)  # the live tokens' slots are all filled
    assert f["idx"].tolist() == [[0, 1, 2, 3]] * 3 and f["counts"].tolist() == [3, 3, 3, 3, 0, 0, 0, 0, 3]


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_order_of_groups_that_hold_the_lowest_value(score):
    """A lone expert at the lowest value counts that (finite), two of them -inf, which a group with nothing does not
    come before."""
    z = torch.zeros(2, 8)
    b = torch.full((8,), LOW)
    b[:2] = -np.inf      # group 0: nothing
    b[4] = -np.inf       # group 2: expert 5 alone
    assert check(z, 2, b, 4, 1, score, False)["idx"].tolist() == [[5, -1]] * 2
    b[4] = LOW
    assert check(z, 2, b, 4, 1, score, False)["idx"].tolist() == [[2, 3]] * 2
    assert check(z, 4, b, 4, 2, score, True)["idx"].tolist() == [[2, 3, 4, 5]] * 2


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k,G,kg", [
    (5, 64, 6, 8, 3), (33, 160, 6, 8, 3), (40, 96, 5, 3, 1), (17, 21, 4, 7, 5), (700, 256, 8, 8, 4), (9, 128, 8, 64, 20),
    (5001, 40, 5, 10, 3),
])
def test_disabled_groups_and_experts(T, E, k, G, kg, dtype, score):
    print("[case] low bias", T, E, k, G, kg, dtype, score, flush=True)
    g = torch.Generator().manual_seed(E)
    b = biases(E, E)
    b.view(G, -1)[torch.rand(G, generator=g) < 0.6] = LOW
    b[torch.rand(E, generator=g) < 0.1] = LOW
    b[torch.rand(E, generator=g) < 0.1] = -np.inf
    for renorm in (False, True):
        check(logits(T, E, T + E, dtype), k, b, G, kg, score, renorm, scale=2.5 if renorm else 1.0)
        check(logits(T, E, T + E, dtype), k, torch.full((E,), LOW), G, kg, score, renorm)
