"""A MoE layer whose experts hold MXFP4 weights: served, and its router and a dense Linear trained.

    python examples/moe_mxfp4.py [--tokens 64] [--hidden 7168] [--ffn 2048] [--experts 32] [--topk 8]

serve() runs the layer as a decode or prompt step does: router, permutation to the experts, both expert
products with E4M3 activations and MXFP4 weights, SwiGLU between them, and the weighted sum back.
train() takes one step of the router (balance loss included) and of a Linear whose three products run in
MXFP4.  The script prints how far both are from the same in float32 on the values the formats hold.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_blockwise_amd as fgb  # noqa: E402


def quantise_experts(w1, w2):
    """Expert weights [E, 2F, H] and [E, H, F] in MXFP4, once."""
    return fgb.mxfp4_quant(w1), fgb.mxfp4_quant(w2)


def serve(x, gate, experts, topk):
    """x bf16 [T, H], gate fp32 [E, H] -> the layer's output bf16 [T, H], the experts chosen and their weights."""
    (w1, s1), (w2, s2) = experts
    idx, weights, counts, _ = fgb.moe_router(x.float() @ gate.t(), topk, renorm=True)
    xq, xs = fgb.fp8_quant_rowwise(x)
    rows, scales, row_map, offsets = fgb.permute_pad(xq, xs, idx, gate.shape[0])
    h = fgb.mxfp4_grouped_gemm(rows, scales, w1, s1, offsets)
    a, a_scales = fgb.swiglu_quant(h, offsets)
    y = fgb.mxfp4_grouped_gemm(a, a_scales, w2, s2, offsets)
    return fgb.unpermute_unpad(y, row_map, weights), idx, weights


class Mxfp4Linear(torch.autograd.Function):
    """y = x w^T with all three products in MXFP4; w's gradient is accumulated in float32."""

    @staticmethod
    def forward(ctx, x, w):
        xq, xs, xqt, xst = fgb.mxfp4_quant_t(x)
        wq, ws, wqt, wst = fgb.mxfp4_quant_t(w)
        ctx.save_for_backward(xqt, xst, wqt, wst)
        return fgb.mxfp4_gemm(xq, xs, wq, ws)

    @staticmethod
    def backward(ctx, dy):
        xqt, xst, wqt, wst = ctx.saved_tensors
        gq, gs, gqt, gst = fgb.mxfp4_quant_t(dy.contiguous())
        return fgb.mxfp4_gemm(gq, gs, wqt, wst), fgb.mxfp4_gemm(gqt, gst, xqt, xst, out_dtype=torch.float32).to(dy.dtype)


class Router(torch.autograd.Function):
    """Logits -> (weights, balance loss); the chosen ids and the slots per expert come beside them."""

    @staticmethod
    def forward(ctx, logits, topk, coef):
        idx, weights, counts, loss = fgb.moe_router(logits, topk, renorm=True, loss_coef=coef)
        ctx.save_for_backward(logits, idx, counts)
        ctx.coef = coef
        ctx.mark_non_differentiable(idx, counts)
        return weights, loss, idx, counts

    @staticmethod
    def backward(ctx, dweights, dloss, *_):
        logits, idx, counts = ctx.saved_tensors
        return fgb.moe_router_backward(logits, idx, counts, dweights.contiguous(), dloss.contiguous(), renorm=True,
                                       loss_coef=ctx.coef), None, None


def train(x, gate, w, topk, coef=0.01):
    """One backward pass: the tokens' chosen weights scale a Linear's output.  Returns the objective and the
    gradients of gate and w."""
    gate, w = gate.detach().requires_grad_(), w.detach().requires_grad_()
    weights, loss, idx, counts = Router.apply(x.float() @ gate.t(), topk, coef)
    y = Mxfp4Linear.apply(x, w)
    objective = (weights[:, :1] * y.float()).square().mean() + loss
    objective.backward()
    return objective.detach(), gate.grad, w.grad, counts


def plain_serve(x, gate, experts, topk):
    """serve() in float32 on the same codes, for comparison."""
    (w1, s1), (w2, s2) = experts
    p = torch.softmax(x.float() @ gate.t(), 1)
    top, idx = p.topk(topk, 1)
    top = top / top.sum(1, keepdim=True)
    xv = fgb.fp8_dequant(*fgb.fp8_quant_rowwise(x), fgb.ROW1x128)
    out = torch.zeros_like(xv)
    for e in range(gate.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = (xv[t] @ fgb.mxfp4_dequant(w1[e], s1[e]).t()).chunk(2, 1)
            a = torch.nn.functional.silu(g) * u
            out.index_add_(0, t, top[t, j, None] * (a @ fgb.mxfp4_dequant(w2[e], s2[e]).t()))
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--ffn", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=8)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = rand(a.tokens, a.hidden).bfloat16()
    gate = rand(a.experts, a.hidden) * a.hidden ** -0.5
    experts = quantise_experts((rand(a.experts, 2 * a.ffn, a.hidden) * a.hidden ** -0.5).bfloat16(),
                               (rand(a.experts, a.hidden, a.ffn) * a.ffn ** -0.5).bfloat16())
    out, idx, weights = serve(x, gate, experts, a.topk)
    ref = plain_serve(x, gate, experts, a.topk)
    print(f"serve: {a.tokens} tokens, relative error {float((out.float() - ref).norm() / ref.norm()):.2e}")
    obj, dgate, dw, counts = train(x, gate, (rand(a.ffn, a.hidden) * a.hidden ** -0.5).bfloat16(), a.topk)
    print(f"train: objective {float(obj):.4f}, |dgate| {float(dgate.norm()):.3e}, |dw| {float(dw.float().norm()):.3e}, "
          f"slots per expert {int(counts[:-1].min())} to {int(counts[:-1].max())}")


if __name__ == "__main__":
    main()
