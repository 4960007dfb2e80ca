"""An infinite gradient in a row of RMSNorm's backward pass: what the formula makes of it, at every width (columns past the
last one belong to lanes that load the last ones once more and must add nothing), and the other rows as if alone."""
import numpy as np
import pytest
import torch

from oracle import norm as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dt,ht", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("cols", [32, 384, 512, 1056, 2080, 4128, 7168, 8224, 16384, 16416])
def test_infinite_gradient(cols, dt, ht):
    import fine_grained_blockwise_amd as fgb
    print("[case] infinite gradient", cols, dt, ht, flush=True)
    g = torch.Generator().manual_seed(cols)
    dy, h = (1e-3 * torch.randn(7, cols, generator=g)).to(dt), torch.randn(7, cols, generator=g).to(ht)
    w = 1 + 0.1 * torch.rand(cols, generator=g)
    for row, col, v in ((1, 0, np.inf), (2, cols - 1, np.inf), (4, cols - 3, -np.inf), (5, cols // 2, -np.inf)):
        dy[row, col] = v
        h[row, col] = 0.5
    h[h == 0] = 1.0
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    with np.errstate(all="ignore"):
        want, wdw = N.backward(dy.double().numpy(), h.double().numpy(), w.double().numpy(), rstd.double().numpy())
    dx, dw = fgb.rmsnorm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV))
    dx, dw = dx.double().cpu().numpy(), dw.double().cpu().numpy()
    for got, ref in ((dx, want), (dw, wdw)):
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(np.isposinf(got), np.isposinf(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    alone = fgb.rmsnorm_backward(dy[3:4].to(DEV), h[3:4].to(DEV), w.to(DEV), rstd[3:4].to(DEV))[0]
    assert np.array_equal(dx[3:4], alone.double().cpu().numpy())
