"""MXFP4 and the router past 32-bit sizes, and inside a HIP graph.  Large outputs are checked at both ends against
the 64-bit reference."""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as O
from oracle import router as R
from test_gpu_mxfp4 import check_product, fgb, same, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print("[case]", *a, flush=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_past_4_gib(dtype):
    rows, cols = (300016, 8192) if dtype == torch.bfloat16 else (140016, 8192)
    say("quant_t", rows, cols, dtype)
    x = torch.empty((rows, cols), dtype=dtype, device=DEV)
    for lo in range(0, rows, 20000):
        x[lo:lo + 20000] = torch.randn((min(20000, rows - lo), cols), device=DEV)
    q, s, qt, st = fgb().mxfp4_quant_t(x)
    q1, s1 = fgb().mxfp4_quant(x)
    for lo in range(0, rows, 50000):  # the same codes from both (compared in pieces)
        assert torch.equal(q[lo:lo + 50000], q1[lo:lo + 50000])
    assert torch.equal(s, s1)
    for r in (0, 12345, rows - 1):
        wq, ws = O.quant(x[r:r + 1].double().cpu().numpy())
        assert same(q[r:r + 1], wq) and same(s[:, r:r + 1], ws)
    for c in (0, cols - 1):
        wq, ws = O.quant(x[:, c].double().cpu().numpy()[None])
        assert same(qt[c:c + 1], wq) and same(st[:, c:c + 1], ws)
    d = fgb().mxfp4_dequant(q, s, out_dtype=dtype)
    for r in (0, rows - 1):
        assert np.array_equal(d[r].double().cpu().numpy(), O.dequant(*O.quant(x[r:r + 1].double().cpu().numpy()))[0])


def test_product_past_4_gib():
    M, N, K = 70000, 32800, 256
    say("gemm", M, N, K)
    x, w = values(M, K, 1, torch.bfloat16), values(N, K, 2, torch.bfloat16)
    a, sa = fgb().mxfp4_quant(x.to(DEV))
    b, sb = fgb().mxfp4_quant(w.to(DEV))
    d = fgb().mxfp4_gemm(a, sa, b, sb)
    for rows in (slice(0, 3), slice(M - 3, M)):
        for cols in (slice(0, 40), slice(N - 40, N)):
            av = O.dequant(*O.quant(x[rows].double().numpy()))
            bv = O.dequant(*O.quant(w[cols].double().numpy()))
            check_product(d[rows, cols], av, bv)


def test_router_past_4_gib():
    T, E, k = 2100032, 520, 4
    say("router", T, E)
    z = torch.empty((T, E), device=DEV)
    for lo in range(0, T, 300000):
        z[lo:lo + 300000] = torch.randn((min(300000, T - lo), E), device=DEV)
    idx, w, counts, loss = fgb().moe_router(z, k, renorm=True, loss_coef=1.0)
    dz = fgb().moe_router_backward(z, idx, counts, w, torch.ones((), device=DEV), renorm=True, loss_coef=1.0)
    assert int(counts[E]) == T and int(counts[:E].sum()) == T * k
    c = counts.cpu().numpy()
    for rows in (slice(0, 4), slice(T - 4, T)):
        zn = z[rows].double().cpu().numpy()
        f = R.forward(zn, k, renorm=True)
        assert np.array_equal(idx[rows].cpu().numpy(), f["idx"])
        assert np.allclose(w[rows].cpu().numpy(), f["weights"], rtol=1e-5, atol=0)
        want = R.backward(zn, f["idx"], c, w[rows].double().cpu().numpy(), 1.0, renorm=True, coef=1.0)
        assert np.abs(dz[rows].double().cpu().numpy() - want).max() <= 16 * 40 * 2.0 ** -24


def test_in_a_graph():
    """Router, experts' products and a training step captured once and replayed on new inputs, each replay against
    the eager result, with eager work and synchronisations between."""
    m = fgb()
    T, H, F, E, k = 40, 512, 256, 8, 2
    x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    z = torch.empty((T, E), device=DEV)
    w1 = m.mxfp4_quant(values(E * 2 * F, H, 3, torch.bfloat16, 1).view(E, 2 * F, H).to(DEV))
    w = values(288, H, 4, torch.bfloat16, 1).to(DEV)
    dy = values(T, 288, 5, torch.bfloat16, 1).to(DEV)

    def fill(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn((T, H), generator=g, device=DEV))
        z.copy_(torch.randn((T, E), generator=g, device=DEV))

    def step():
        idx, wt, counts, loss = m.moe_router(z, k, renorm=True, loss_coef=0.1)
        dz = m.moe_router_backward(z, idx, counts, wt, loss, renorm=True, loss_coef=0.1)
        rows, scales, row_map, offs = m.permute_pad(*m.fp8_quant_rowwise(x), idx, E)
        h = m.mxfp4_grouped_gemm(rows, scales, *w1, offs, d=torch.zeros((rows.shape[0], 2 * F), dtype=torch.bfloat16,
                                                                        device=DEV))
        xq, xs, xqt, xst = m.mxfp4_quant_t(x)
        wq, ws, wqt, wst = m.mxfp4_quant_t(w)
        gq, gs, gqt, gst = m.mxfp4_quant_t(dy)
        return [idx, wt, counts, loss, dz, h, m.mxfp4_gemm(xq, xs, wq, ws), m.mxfp4_gemm(gq, gs, wqt, wst),
                m.mxfp4_gemm(gqt, gst, xqt, xst, out_dtype=torch.float32), m.mxfp4_dequant(xq, xs)]

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(1, 5):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
