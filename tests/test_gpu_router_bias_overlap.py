"""The bias's update into a buffer that lies over a part of the bias."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("E", [2, 64, 65, 300, 1024])
@pytest.mark.parametrize("shift", [-70, -64, -1, 1, 64, 70])
def test_update_into_an_overlapping_buffer(E, shift):
    import fine_grained_blockwise_amd as f
    g = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 100, (E + 1,), generator=g, dtype=torch.int32).to(DEV)
    buf = torch.randn(E + 140, generator=g).to(DEV)
    bias, out = buf[70: 70 + E], buf[70 + shift: 70 + shift + E]
    want = f.moe_bias_update(bias.clone(), counts, 1e-3)
    f.moe_bias_update(bias, counts, 1e-3, out=out)
    assert torch.equal(out, want)
