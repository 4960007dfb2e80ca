"""The places that an output of the norm and its gradient may take, at every width: bit for bit what an output of its own
gets; what overlaps otherwise is refused through the binding, too."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def tensors(rows, cols, *types):
    g = torch.Generator().manual_seed(cols)
    return [torch.randn(rows, cols, generator=g).to(t).to(DEV) for t in types]


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(2100, 96), (2100, 1536), (530, 7168), (300, 8224), (270, 20480)])
def test_forward_in_place(rows, cols, t):
    """h over x; y over x and over the residual (through the C entry point, as the binding allocates y)."""
    f = fgb()
    code = f.F32 if t == F32 else f.BF16
    x, r = tensors(rows, cols, t, t)
    w = torch.rand(cols, generator=torch.Generator().manual_seed(1)).to(DEV)
    want = f.rmsnorm_quant(x, w, residual=r, group=32, y_dtype=t)
    a = x.clone()
    got = f.rmsnorm_quant(a, w, residual=r, group=32, y_dtype=t, h=a)
    assert got[3] is a and all(torch.equal(p, q) for p, q in zip(want, got))
    for k in range(2):
        v, h, rstd = [x.clone(), r.clone()], torch.empty_like(x), torch.empty(rows, device=DEV)
        f._call("rmsnorm_quant", v[0].data_ptr(), code, rows, cols, cols, v[1].data_ptr(), code, cols, w.data_ptr(), f.F32,
                1e-6, 32, h.data_ptr(), cols, rstd.data_ptr(), None, None, v[k].data_ptr(), code, cols, f._stream(x))
        assert torch.equal(v[k], want[2]) and torch.equal(h, want[3]) and torch.equal(rstd, want[4])


@pytest.mark.parametrize("rows,cols", [(2100, 96), (2100, 1536), (530, 7168), (300, 8224), (270, 20480)])
def test_gradient_over_h(rows, cols):
    f = fgb()
    dy, h, dh = tensors(rows, cols, BF16, BF16, BF16)
    w = torch.rand(cols, generator=torch.Generator().manual_seed(1)).to(DEV)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    want = f.rmsnorm_backward(dy, h, w, rstd, dh=dh)
    a = h.clone()
    got = f.rmsnorm_backward(dy, a, w, rstd, dh=dh, dx=a)
    assert got[0] is a and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_columns_of_one_buffer_and_refusals():
    f = fgb()
    x, r = tensors(70, 256, BF16, BF16)
    w = torch.ones(256, device=DEV)
    want = f.rmsnorm_quant(x, w, residual=r)
    wide = torch.full((70, 1024), 7.0, dtype=BF16, device=DEV)
    xv, rv, hv = wide[:, :256], wide[:, 256:512], wide[:, 520:776]
    xv.copy_(x)
    rv.copy_(r)
    got = f.rmsnorm_quant(xv, w, residual=rv, h=hv)
    assert all(torch.equal(p, q) for p, q in zip(want, got) if p is not None)
    assert (wide[:, 512:520] == 7).all() and (wide[:, 776:] == 7).all() and torch.equal(xv, x) and torch.equal(rv, r)
    for bad in (wide[:, 248:504], wide[:, 504:760], wide.view(-1)[256: 256 + 70 * 256].view(70, 256)):
        with pytest.raises(RuntimeError, match="lies over"):
            f.rmsnorm_quant(xv, w, residual=rv, h=bad)
    with pytest.raises(RuntimeError, match="lies over"):
        f.rmsnorm_quant(x[:-1], w, residual=r[:-1], h=r[1:])
    rstd = torch.ones(70, device=DEV)
    buf = torch.empty(72 * 256, dtype=BF16, device=DEV)
    dy = buf[: 70 * 256].view(70, 256)
    for dx in (buf[256: 71 * 256].view(70, 256), buf[8: 70 * 256 + 8].view(70, 256)):
        with pytest.raises(RuntimeError, match="dx lies over dy"):
            f.rmsnorm_backward(dy, x, w, rstd, dx=dx)
    n = f.rmsnorm_backward_workspace_size(70, 256)
    room = torch.zeros(n + 70 * 512, dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError, match="workspace lies over dh"):
        f.rmsnorm_backward(dy, x, w, rstd, dh=room[: 70 * 512].view(BF16).view(70, 256), workspace=room[:n])
