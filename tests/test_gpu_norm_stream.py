"""The stream that rmsnorm_quant returns without a residual is the caller's tensor, however its rows lie."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["usual", "slice", "misaligned", "every other column", "transposed", "one row"])
def test_stream_without_a_residual_is_x(kind):
    import fine_grained_blockwise_amd as f
    base = torch.randn(12, 640, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    x = dict(usual=base, slice=base[:, 128:384], misaligned=base[:, 3:259], transposed=base[:, :32].t().contiguous().t(),
             **{"every other column": base[:, :512:2], "one row": base[4:5, 5:261]})[kind]
    h = f.rmsnorm_quant(x, torch.ones(x.shape[1], device=DEV), group=32)[3]
    assert h is x
    h.add_(1.0)
    assert torch.equal(h, x)
