"""Clipping by a norm that FP32, in which it is returned, does not hold."""
import math

import pytest
import torch

from test_gpu_grads import fgb

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
MOST = torch.finfo(F32).max


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_norm_that_is_returned_as_infinite_clips_nothing(t, given, in_place):
    """Finite gradients whose norm is 1.6e40: the caller sees inf, so the gradients are scaled only."""
    g = [torch.full((3000,), 3e38, dtype=t, device=DEV), torch.full((5,), -2.0, dtype=t, device=DEV)]
    want = [(v.float() * 0.25).to(t) for v in g]
    out = None if in_place else [torch.empty_like(v) for v in g]
    s = fgb().grad_sumsq(g) if given else None
    norm = fgb().grad_clip(g, 1.0, scale=0.25, out=out, sumsq=s)
    assert float(norm) == math.inf
    assert all(torch.equal(a, b) for a, b in zip(g if in_place else out, want))


def test_the_norm_nearest_to_the_border():
    """2^128 - 2^103 is where FP32 rounds to infinity: just below it the norm is the largest number, and clips."""
    for n, inf in ((MOST + 2.0 ** 102, False), (MOST + 2.0 ** 104, True)):
        g = [torch.tensor([MOST, 1e30], device=DEV)]
        s = torch.tensor(n * n, dtype=torch.float64, device=DEV)
        norm = fgb().grad_clip(g, MOST / 2, sumsq=s)
        assert float(norm) == (math.inf if inf else MOST)
        assert float(g[0][1]) == pytest.approx(1e30 if inf else 5e29, rel=1e-6)
