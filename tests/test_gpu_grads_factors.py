"""Clipping by factors that FP32 holds as subnormals or not at all.  Bounds as in test_gpu_grads.py."""
import pytest
import torch

from test_gpu_grads import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("most", [1e-1, 1e-3, 1e-9, 1e-25, 1e-37])
def test_factors_below_fp32_s_normal_range(t, most):
    g = [torch.tensor([3e38], device=DEV).to(t), torch.linspace(-1e36, 1e36, 3001, device=DEV).to(t)]
    check([v.clone() for v in g], most, 1.0, [F32, BF16])
    check([v.clone() for v in g], most, in_place=True)


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-38, 1e-42, 1e-60, 1e38, 1e45, 1e60])
def test_scales_outside_fp32(t, scale):
    """What is left of 1 / scale and 0, which an infinite factor would make NaN."""
    g = [torch.tensor([1.0, -3.0, 0.0, 0.7] * 9, device=DEV).mul(min(1 / scale, 1e37)).to(t)]
    check([v.clone() for v in g], 1e30, scale, [F32])
    check([v.clone() for v in g], 1e-3, scale, [BF16])
    check([v.clone() for v in g], 1e30, scale, in_place=True)
