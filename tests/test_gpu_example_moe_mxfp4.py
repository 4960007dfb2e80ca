"""The example's layer: served against float32 on the same codes, trained against autograd through plain torch.
The served output passes through one E4M3 rounding (the SwiGLU's, half a step of 2^-3: at most 2^-4 of an element,
random over a sum) and BF16 roundings: its relative error in the 2-norm is below 2^-4."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_mxfp4.py")
    spec = importlib.util.spec_from_file_location("moe_mxfp4", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rand(g, *s):
    return torch.randn(s, generator=g, device=DEV)


@pytest.mark.parametrize("tokens", [1, 7, 300])
def test_serve(tokens):
    m = example()
    g = torch.Generator(device=DEV).manual_seed(tokens)
    H, F, E, k = 512, 256, 8, 3
    x, gate = rand(g, tokens, H).bfloat16(), rand(g, E, H) * H ** -0.5
    experts = m.quantise_experts((rand(g, E, 2 * F, H) * H ** -0.5).bfloat16(), (rand(g, E, H, F) * F ** -0.5).bfloat16())
    out, idx, weights = m.serve(x, gate, experts, k)
    ref = m.plain_serve(x, gate, experts, k)
    assert float((out.float() - ref).norm() / ref.norm()) < 2 ** -4
    assert bool((weights.sum(1) - 1).abs().max() < 1e-5)


def test_train():
    """The gradients against autograd of the same objective on the values the formats hold."""
    m = example()
    fgb = m.fgb
    g = torch.Generator(device=DEV).manual_seed(3)
    T, H, F, E, k, coef = 160, 256, 96, 8, 2, 0.02
    x, gate, w = rand(g, T, H).bfloat16(), rand(g, E, H) * H ** -0.5, (rand(g, F, H) * H ** -0.5).bfloat16()
    obj, dgate, dw, counts = m.train(x, gate, w, k, coef)
    gr = gate.clone().requires_grad_()
    p = torch.softmax(x.float() @ gr.t(), 1)
    top, idx = p.topk(k, 1)
    weights = top / top.sum(1, keepdim=True)
    c = torch.bincount(idx.reshape(-1), minlength=E)
    assert torch.equal(c.int(), counts[:-1])
    loss = coef * E / (k * T * T) * (c.float() * p.sum(0)).sum()
    value = lambda t: fgb.mxfp4_dequant(*fgb.mxfp4_quant(t))  # noqa: E731
    y = (value(x) @ value(w).t()).bfloat16().float().requires_grad_()
    ref = (weights[:, :1] * y).square().mean() + loss
    ref.backward()
    ref = float(ref.detach())
    assert abs(float(obj) - ref) <= 1e-5 * abs(ref)
    assert float((dgate - gr.grad).norm() / gr.grad.norm()) < 1e-3  # y is BF16 on both sides, rounded apart
    dy = y.grad.bfloat16()
    want = value(dy.t().contiguous()) @ value(x.t().contiguous()).t()
    assert float((dw.float() - want).norm() / want.norm()) < 2 ** -7  # dw returned in BF16, dy's codes near ties
