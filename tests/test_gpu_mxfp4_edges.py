"""Ties, subnormals, the largest values, infinities and NaN through every MXFP4 quantizer: FP32 and BF16, the rows
of mxfp4_quant, and the rows and the columns of mxfp4_quant_t, against the 64-bit reference bit for bit."""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def neighbours(v, dtype):
    """float32 values and the numbers of `dtype` next to them on either side (magnitudes)."""
    step = 1 if dtype == torch.float32 else 1 << 16
    bits = v.view(np.int32)
    return [v, np.where(v > 0, bits + step, bits).view(np.float32), np.where(v > 0, bits - step, bits).view(np.float32)]


def groups(dtype):
    """Groups of 32: every E2M1 value and tie and its neighbours at many exponents, both signs, then extremes."""
    m = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    low = -149 if dtype == torch.float32 else -133
    rows = []
    for e in (low, low + 3, low + 6, -130, -128, -127, -126, -125, -124, -60, -2, 0, 1, 60, 124):
        v = np.ldexp(m, e).astype(np.float32)
        if dtype == torch.bfloat16:
            v = (v.view(np.int32) & ~0xFFFF).view(np.float32)  # (below the least exponents not all are BF16)
        for w in neighbours(v, dtype):
            rows.append(np.concatenate([w, [0.0], -w, [-0.0]]))
            rows.append(np.concatenate([w[:9], np.zeros(14), -w[:9]]))  # the largest is not 6 times a power of two
    top = np.float32(np.finfo(np.float32).max) if dtype == torch.float32 else np.int32(0x7F7F0000).view(np.float32)
    rows += [np.full(32, top), np.r_[top, np.zeros(31)], np.r_[np.inf, np.ones(31)], np.r_[np.ones(31), np.nan],
             np.r_[-np.inf, np.nan, np.zeros(30)], np.zeros(32)]
    return np.stack(rows).astype(np.float32)


def same(q, s, wq, ws, n):
    q, s = q.cpu().numpy()[:n], s.cpu().numpy()[:, :n]
    assert np.array_equal(s, ws)
    fine = O.row_scales(ws, 1)[:, 0] != 255  # (a NaN group's codes mean nothing)
    assert np.array_equal(q[fine], wq[fine])


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_quantizer_at_the_edges(dtype, rule):
    import fine_grained_blockwise_amd as m
    x = groups(dtype)
    t = torch.from_numpy(x).to(dtype)
    assert np.array_equal(t.float().numpy(), x, equal_nan=True)
    q, s = O.quant(x, rule)
    n = len(x)
    same(*m.mxfp4_quant(t.to(DEV), rule=rule), q, s, n)
    same(*m.mxfp4_quant_t(t.to(DEV), rule=rule)[:2], q, s, n)
    cols = torch.zeros((32, (n + 31) // 32 * 32), dtype=dtype)
    cols[:, :n] = t.t()
    same(*m.mxfp4_quant_t(cols.to(DEV), rule=rule)[2:], q, s, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,rows,cols", [(3, 45, 96), (5, 300, 288), (40, 257, 1056)])
def test_stacks_are_their_matrices(G, rows, cols, dtype):
    import fine_grained_blockwise_amd as m
    x = torch.randn((G, rows, cols), generator=torch.Generator().manual_seed(G)).to(dtype).to(DEV)
    alone = [m.mxfp4_quant_t(x[g]) for g in range(G)]
    for got in (m.mxfp4_quant(x), m.mxfp4_quant_t(x)):
        for i, t in enumerate(got):
            assert all(torch.equal(t[g], alone[g][i]) for g in range(G))
    wq, ws = O.quant(x[G - 1].double().cpu().numpy())
    assert np.array_equal(alone[-1][0].cpu().numpy(), wq) and np.array_equal(alone[-1][1].cpu().numpy(), ws)
