"""Ids outside the experts in the router's gradient: such slots are ignored, and every row is written, renormed or not."""
import pytest
import torch

from oracle import router as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [7, 64, 300, 1024])
def test_rows_whose_ids_are_no_experts(E, renorm, score):
    """The loss's part alone: what the forward's ids give without gradients of the weights."""
    import fine_grained_blockwise_amd as f
    T, k = 37, 3
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).to(DEV)
    idx, _, counts, _ = f.moe_router(z, k, score=score, renorm=renorm, loss_coef=0.1)
    one = torch.ones((), device=DEV)
    want = f.moe_router_backward(z, idx, counts, None, one, score=score, renorm=renorm, loss_coef=0.1)
    bad = idx.clone()
    bad[::2] = E
    bad[4] = 2 ** 31 - 1
    dw = torch.ones(T, k, device=DEV)
    dz = torch.full((T, E), 7.0, device=DEV)
    f._call("moe_router_backward", z.data_ptr(), f.F32, T, E, E, k, bad.data_ptr(), counts.data_ptr(), dw.data_ptr(),
            one.data_ptr(), score, int(renorm), 1.0, 0.1, dz.data_ptr(), E, f._stream(z))
    # (no larger than 0.1 E / k: p and the sum of g p within 32 roundings each on either side)
    assert ((dz[::2] - want[::2]).abs() <= 64 * 2.0 ** -24 * 0.1 * E / k).all()
