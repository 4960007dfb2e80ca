"""The norm, the grouped router, the experts' products, both gradients, the bias's update and clipping as one step uses
them: against the 64-bit references, captured in a graph, and on several streams at once.

Gradient bounds: the router's gradient of each logit is within 16 (r + 28) u of the largest |g| and |D| (r the logits'
range, u = 2^-24); through y = logits' input it grows by sum |gate|, and the norm's gradient maps an error e of dy to at
most rstd (|w| e + |hat| mean(|hat| |w| e)); the norm's own error is test_gpu_norm.py's."""
import threading

import numpy as np
import pytest
import torch

from oracle import norm as N
from oracle import router as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
T, H, F, E, K, G, KG = 203, 512, 256, 32, 4, 8, 3
HOW = dict(score=R.SIGMOID, renorm=True, scale=2.5, loss_coef=0.01)


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, sc=1.0: torch.randn(*s, generator=g) * sc  # noqa: E731
    return dict(x=n(T, H).to(BF16), r=n(T, H, sc=2.0).to(BF16), w=(1 + n(H, sc=0.2)).to(BF16), gate=n(E, H, sc=H ** -0.5),
                bias=n(E, sc=0.05), w1=n(E, 2 * F, H, sc=0.05).to(BF16), w2=n(E, H, F, sc=0.05).to(BF16),
                dweights=n(T, K, sc=1e-2), dloss=torch.ones(()), dh=n(T, H, sc=1e-3).to(BF16))


def step(I, ws):
    """One pass; every output by name.  ws: workspaces of the router, permute_pad, the norm's gradient and clipping."""
    f = fgb()
    q, s, y, h, rstd = f.rmsnorm_quant(I["x"], I["w"], residual=I["r"], y_dtype=F32)
    logits = y @ I["gate"].t()
    idx, weights, counts, loss = f.moe_router(logits, K, bias=I["bias"], groups=G, topk_groups=KG, workspace=ws[0], **HOW)
    rows, scales, row_map, offsets = f.permute_pad(q, s, idx, E, 16, T * K + 15 * E, ws[1])
    w1q, w1s = f.fp8_quant_blockwise_t(I["w1"])[:2]
    w2q, w2s = f.fp8_quant_blockwise_t(I["w2"])[:2]
    a, a_s = f.swiglu_quant(f.fp8_grouped_gemm(rows, scales, w1q, w1s, offsets), offsets)
    out = f.unpermute_unpad(f.fp8_grouped_gemm(a, a_s, w2q, w2s, offsets), row_map, weights)
    dz = f.moe_router_backward(logits, idx, counts, I["dweights"], I["dloss"], **HOW)
    dy = dz @ I["gate"]
    dx, dw = f.rmsnorm_backward(dy, h, I["w"], rstd, dh=I["dh"], workspace=ws[2])
    grads = [dw, dz.t() @ y]
    clipped = [torch.empty_like(g) for g in grads]
    norm = f.grad_clip(grads, 1e-2, out=clipped, workspace=ws[3])
    bias = f.moe_bias_update(I["bias"], counts, 1e-3)
    return dict(q=q, s=s, y=y, h=h, rstd=rstd, logits=logits, idx=idx, weights=weights, counts=counts, loss=loss, out=out,
                dz=dz, dy=dy, dx=dx, dw=dw, dgate=grads[1], norm=norm, cw=clipped[0], cg=clipped[1], bias=bias)


def workspaces():
    f = fgb()
    sizes = (f.moe_router_workspace_size(T, E), f.permute_pad_workspace_size(T, K, E), f.rmsnorm_backward_workspace_size(T, H),
             f.grad_sumsq_workspace_size([H, E * H]))
    return [torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes]


def on_gpu(I):
    return {k: v.to(DEV) for k, v in I.items()}


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.int16).numpy() if t.dtype == BF16 else t.view(torch.int32).numpy() if t.dtype == F32 else t.numpy()


def d(t):
    return t.detach().double().cpu().numpy()


def test_step_against_the_references():
    I = inputs(0)
    o = step(on_gpu(I), workspaces())
    h = (I["x"].float() + I["r"].float()).to(BF16)
    assert torch.equal(o["h"].cpu(), h)
    wy, wr = N.forward(d(h), d(I["w"]), 1e-6)
    assert (np.abs(d(o["y"]) - wy) <= 38 * U * np.abs(wy)).all() and (np.abs(d(o["rstd"]) - wr) <= 36 * U * wr).all()
    q, s = fgb().fp8_quant_rowwise(o["y"])
    assert torch.equal(o["q"], q) and torch.equal(o["s"], s)
    z = d(o["logits"])
    idx = R.choose(z, K, R.SIGMOID, I["bias"].numpy(), G, KG)
    f = R.forward(z, K, R.SIGMOID, True, 2.5, 0.01, idx=idx)
    assert np.array_equal(o["idx"].cpu().numpy(), idx) and np.array_equal(o["counts"].cpu().numpy(), f["counts"])
    tol = (z.max() - z.min() + 28) * U
    assert (np.abs(d(o["weights"]) - f["weights"]) <= 4 * tol * f["weights"]).all()
    assert abs(float(o["loss"]) - f["loss"]) <= 4 * tol * f["loss"]
    # the experts read the norm's codes: the same output from the quantiser's codes of y
    f2 = fgb()
    Id = on_gpu(I)
    rows, scales, row_map, off = f2.permute_pad(q, s, o["idx"], E, 16)
    w1q, w1s = f2.fp8_quant_blockwise_t(Id["w1"])[:2]
    w2q, w2s = f2.fp8_quant_blockwise_t(Id["w2"])[:2]
    a, a_s = f2.swiglu_quant(f2.fp8_grouped_gemm(rows, scales, w1q, w1s, off), off)
    assert torch.equal(o["out"], f2.unpermute_unpad(f2.fp8_grouped_gemm(a, a_s, w2q, w2s, off), row_map, o["weights"]))
    # gradients, each from what the step handed on
    dz = R.backward(z, idx, f["counts"], d(I["dweights"]), 1.0, R.SIGMOID, True, 2.5, 0.01)
    n = int(f["counts"][E])
    big = 0.01 * E / (K * n * n) * f["counts"][:E].max() + 2.5 * np.abs(d(I["dweights"])).max()
    ez = 16 * tol * big
    assert (np.abs(d(o["dz"]) - dz) <= ez).all()
    gate = d(I["gate"])
    dy = dz @ gate
    ey = ez * np.abs(gate).sum(0)[None] + E * U * (np.abs(dz) @ np.abs(gate))
    dx, dw = N.backward(dy, d(h), d(I["w"]), d(o["rstd"]), d(I["dh"]))
    r, w = d(o["rstd"])[:, None], np.abs(d(I["w"]))[None]
    hat = np.abs(d(h) * r)
    a = np.abs(dy) * w
    ex = r * (w * ey + hat * (hat * w * ey).mean(1, keepdims=True))
    ex += r * (4 * U * a + 70 * U * hat * (a * hat).mean(1, keepdims=True)) + 2 * U * (np.abs(dx) + np.abs(d(I["dh"])))
    assert (np.abs(d(o["dx"]) - dx) <= ex + 2.0 ** -8 * (np.abs(dx) + ex)).all()
    assert (np.abs(d(o["dw"]) - dw) <= (ey * hat).sum(0) + (T / 512 + 100) * U * (np.abs(dy) * hat).sum(0)).all()
    norm = np.sqrt((d(o["dw"]) ** 2).sum() + (d(o["dgate"]) ** 2).sum())
    assert abs(float(o["norm"]) - norm) <= (2.0 ** -24 + 1e-12) * norm and norm > 1e-2
    for c, g in ((o["cw"], o["dw"]), (o["cg"], o["dgate"])):
        assert (np.abs(d(c) - d(g) * (1e-2 / norm)) <= (2 * U + 1e-9) * np.abs(d(g)) * (1e-2 / norm) + 2.0 ** -149).all()
    want = I["bias"] + 1e-3 * torch.from_numpy(np.sign(f["counts"][:E].sum() - f["counts"][:E].astype(np.int64) * E)).float()
    assert torch.equal(o["bias"].cpu(), want)


def test_step_in_a_graph():
    """Captured once and replayed on new inputs, with eager passes and synchronisations between: bit for bit the same;
    a second graph of the same step shares the first one's workspaces."""
    ws = workspaces()
    static = on_gpu(inputs(0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(static, ws)
        graphs.append((graph, got))
    for rep in range(4):
        new = inputs(10 + rep)
        for k, v in new.items():
            static[k].copy_(v.to(DEV))
        torch.cuda.synchronize()
        graph, got = graphs[rep % 2]
        graph.replay()
        torch.cuda.synchronize()
        have = {k: bits(v) for k, v in got.items()}
        want = step(on_gpu(new), workspaces())
        torch.cuda.synchronize()
        for k, v in want.items():
            assert np.array_equal(have[k], bits(v)), (rep, k)


def test_steps_on_several_streams_at_once():
    ins = [on_gpu(inputs(20 + i)) for i in range(4)]
    torch.cuda.synchronize()
    got, fails, barrier = [None] * 4, [], threading.Barrier(4)

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                barrier.wait()
                o = step(ins[i], workspaces())
            stream.synchronize()
            got[i] = {k: bits(v) for k, v in o.items()}
        except BaseException as e:  # noqa: B902
            fails.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails, fails
    for i in range(4):
        for k, v in step(ins[i], workspaces()).items():
            assert np.array_equal(got[i][k], bits(v)), (i, k)


def test_workspaces_that_are_too_small_or_elsewhere():
    f, I = fgb(), on_gpu(inputs(1))
    y, h, rstd = f.rmsnorm_quant(I["x"], I["w"], residual=I["r"], y_dtype=F32)[2:]
    for ws in (torch.empty(8, dtype=torch.uint8, device=DEV), torch.empty(0, dtype=torch.uint8, device=DEV)):
        with pytest.raises(RuntimeError, match="workspace"):
            f.rmsnorm_backward(y, h, I["w"], rstd, workspace=ws)
        with pytest.raises(RuntimeError, match="workspace"):
            f.grad_clip([y], 1.0, workspace=ws)
        with pytest.raises(RuntimeError, match="workspace"):
            f.moe_router(y, K, bias=torch.zeros(H, device=DEV), workspace=ws)
    with pytest.raises(ValueError, match="GPU"):
        f.grad_sumsq([y], workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        f.rmsnorm_backward(y, h, I["w"], rstd, workspace=torch.empty(1 << 22, dtype=torch.uint8))
