"""RMSNorm into FP8 and its gradient on the GPU against the 64-bit reference.

With u = 2^-24: a sum of squares passes through at most 64 roundings (products, a lane's 32 values, the lanes and
waves of a row), all of positive terms, so rstd is within 36 u (half of 64, and 4 for the mean, eps, the root and the
division) and y within 38 u of y.  The stream h is the FP32 sum rounded to its type: exact.  Codes and scales are
those that fp8_quant_rowwise gives for the FP32 y, bit for bit.

Gradient: mean(a hat) is within 67 u of M = mean |a hat| (its terms' three roundings among them), so dx is within
rstd (4 u |a| + 70 u |hat| M) + 2 u (|dx| + |dh|), and a rounding to its type; dweight within
(rows / 512 + 100) u sum |dy hat|: a part's rows in turn, then the parts."""
import numpy as np
import pytest
import torch

from oracle import norm as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def half_step(t):
    return torch.finfo(t).eps / 2


def rows_of(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * std * torch.exp(0.7 * torch.randn((shape[0], 1), generator=g))
    x[:, : max(1, shape[1] // 64)] *= 20
    return x.to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def check_forward(x, w, r, group, y_dtype, eps=1e-6, quant=True, dev=None):
    """x, w, r: CPU tensors; dev: the GPU tensors to use in their place."""
    xd, wd, rd = dev or (x.to(DEV), w.to(DEV), None if r is None else r.to(DEV))
    q, s, y, h, rstd = fgb().rmsnorm_quant(xd, wd, residual=rd, eps=eps, group=group, quant=quant, y_dtype=y_dtype)
    want_h = x if r is None else (x.float() + r.float()).to(r.dtype)
    assert torch.equal(h.cpu(), want_h) and h.dtype == want_h.dtype
    wy, wr = N.forward(np64(want_h), np64(w), eps)
    assert (np.abs(np64(rstd) - wr) <= 36 * U * wr).all()
    y32 = fgb().rmsnorm_quant(h, wd, eps=eps, quant=False, y_dtype=F32)[2]
    lim = 38 * U * np.abs(wy) + 2.0 ** -149
    assert (np.abs(np64(y32) - wy) <= lim).all()
    if y_dtype is not None:
        assert torch.equal(y, y32.to(y_dtype))
    else:
        assert y is None
    if quant:
        wq, ws = fgb().fp8_quant_rowwise(y32, group)
        assert torch.equal(q, wq) and torch.equal(s, ws)
    else:
        assert q is None and s is None
    return h, rstd


@pytest.mark.parametrize("xt,rt,wt,yt", [
    (BF16, BF16, BF16, None), (BF16, F32, F32, BF16), (F32, BF16, BF16, F32), (F32, F32, BF16, BF16),
    (BF16, None, F32, F32), (F32, None, BF16, None),
])
@pytest.mark.parametrize("rows,cols,group", [
    (1, 128, 128), (2, 32, 32), (3, 1024, 128), (5, 1056, 32), (4, 2048, 128), (7, 2080, 32), (1, 4096, 128),
    (9, 4224, 128), (3, 7168, 128), (2, 8192, 32), (2, 8224, 32), (1, 16384, 128), (2, 16512, 128), (1, 32768, 128),
    (700, 256, 128), (41, 512, 32),
])
def test_forward(rows, cols, group, xt, rt, wt, yt):
    print("[case] rmsnorm_quant", rows, cols, group, xt, rt, wt, yt, flush=True)
    x = rows_of((rows, cols), rows + cols, xt)
    r = None if rt is None else rows_of((rows, cols), rows + cols + 1, rt, 2.0)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(wt)
    check_forward(x, w, r, group, yt)


@pytest.mark.parametrize("rows,cols", [(4097, 7168), (16390, 544)])
def test_forward_many_rows(rows, cols):
    print("[case] rmsnorm_quant", rows, cols, flush=True)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(BF16)
    check_forward(rows_of((rows, cols), 1, BF16), w, rows_of((rows, cols), 2, BF16, 2.0), 32, None)


def test_forward_without_codes_takes_columns_that_no_group_divides():
    w = torch.ones(96, dtype=F32)
    check_forward(rows_of((5, 96), 1, BF16), w, None, 128, BF16, quant=False)


def test_forward_zero_rows_and_tiny_values():
    x = rows_of((6, 256), 5, F32)
    x[1] = 0
    x[2] *= 1e-18
    x[3, 128:] = 0  # a group of zeros
    x[4] *= 1e16
    check_forward(x, torch.ones(256), None, 128, F32)
    check_forward(x, torch.ones(256), torch.zeros(6, 256), 32, F32, eps=1e-5)
    q, s, y, h, rstd = fgb().rmsnorm_quant(x[1:2].to(DEV), torch.ones(256, device=DEV), y_dtype=F32, eps=0.25)
    assert float(rstd) == 2.0 and not q.any() and (s == 127 - 22).all() and not y.any()


def test_forward_nan_rows_stay_alone():
    x = rows_of((5, 384), 6, BF16)
    x[2, 7] = float("nan")
    x[3, 300] = float("inf")
    w = torch.ones(384, dtype=BF16)
    q, s, y, h, rstd = fgb().rmsnorm_quant(x.to(DEV), w.to(DEV), y_dtype=F32)
    keep = [0, 1, 4]
    wy, _ = N.forward(np64(x[keep]), np64(w), 1e-6)
    assert (np.abs(np64(y)[keep] - wy) <= 38 * U * np.abs(wy)).all()
    assert torch.isnan(y[2]).all() and torch.isnan(rstd[2]) and torch.isnan(y[3, 300])


def test_forward_strides_and_alignment():
    base = rows_of((12, 640), 7, BF16).to(DEV)
    turned = rows_of((256, 12), 8, BF16).to(DEV).t()
    weights = (1 + 0.3 * torch.randn(300, generator=torch.Generator().manual_seed(3))).to(BF16).to(DEV)
    cases = [base[:, 128:384], base[::2, :256], base[:, 3:259], base[:, :512:2], turned, base[4:5, 5:261]]
    for i, x in enumerate(cases):
        print("[case] strides", i, flush=True)
        w = weights[i: i + 256]
        r = rows_of(x.shape, i, F32).to(DEV)
        check_forward(x.cpu(), w.cpu(), r.cpu(), 128, BF16, dev=(x, w, r))
        check_forward(r.cpu(), w.cpu(), x.cpu(), 128, BF16, dev=(r, w, x))


def test_forward_into_the_residual():
    x, r = rows_of((33, 1024), 1, BF16), rows_of((33, 1024), 2, F32)
    w = torch.ones(1024)
    pad = torch.full((33, 1056), 7.0, device=DEV)
    view = pad[:, :1024]
    view.copy_(r)
    a = fgb().rmsnorm_quant(x.to(DEV), w.to(DEV), residual=r.to(DEV))
    b = fgb().rmsnorm_quant(x.to(DEV), w.to(DEV), residual=view, h=view)
    assert b[3] is view and all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
    assert (pad[:, 1024:] == 7).all()


def test_forward_no_rows():
    q, s, y, h, rstd = fgb().rmsnorm_quant(torch.empty(0, 256, device=DEV), torch.ones(256, device=DEV), y_dtype=BF16)
    assert q.shape == (0, 256) and s.shape == (0, 2) and y.shape == (0, 256) and rstd.shape == (0,)


# ---- gradient -------------------------------------------------------------------------------

def check_backward(dy, h, w, dh, dev=None, dx=None):
    dyd, hd, wd, dhd = dev or (dy.to(DEV), h.to(DEV), w.to(DEV), None if dh is None else dh.to(DEV))
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    got, dw = fgb().rmsnorm_backward(dyd, hd, wd, rstd.to(DEV), dh=dhd, dx=dx)
    assert got.dtype == h.dtype and dw.dtype == F32
    a, b = np64(dy) * np64(w), np64(h) * np64(rstd)[:, None]
    want, wdw = N.backward(np64(dy), np64(h), np64(w), np64(rstd), None if dh is None else np64(dh))
    M = np.abs(a * b).mean(1, keepdims=True) if h.shape[0] else 0.0
    lim = np64(rstd)[:, None] * (4 * U * np.abs(a) + 70 * U * np.abs(b) * M)
    lim += 2 * U * (np.abs(want) + (0 if dh is None else np.abs(np64(dh)))) + 2.0 ** -149
    if h.dtype == BF16:
        lim += half_step(BF16) * (np.abs(want) + lim) + 2.0 ** -134
    assert (np.abs(np64(got) - want) <= lim).all()
    deep = (h.shape[0] / 512 + 100) * U
    assert (np.abs(np64(dw) - wdw) <= deep * np.abs(np64(dy) * b).sum(0) + 2.0 ** -140).all()
    return got, dw


@pytest.mark.parametrize("dt,ht,wt,add", [
    (BF16, BF16, BF16, True), (BF16, F32, F32, True), (F32, BF16, BF16, False), (F32, F32, BF16, True),
])
@pytest.mark.parametrize("rows,cols", [
    (1, 32), (2, 128), (5, 1024), (3, 1056), (9, 2048), (7, 2080), (1, 4096), (6, 4128), (3, 7168), (2, 8192), (2, 8224),
    (3, 16384), (1, 16416), (2, 32768), (701, 96), (515, 2144),
])
def test_backward(rows, cols, dt, ht, wt, add):
    print("[case] rmsnorm_backward", rows, cols, dt, ht, wt, add, flush=True)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(wt)
    check_backward(rows_of((rows, cols), 1, dt, 1e-3), rows_of((rows, cols), 2, ht),
                   w, rows_of((rows, cols), 3, ht, 1e-3) if add else None)


@pytest.mark.parametrize("rows,cols", [(2049, 512), (4099, 7168), (8195, 64), (2500, 1536), (519, 8224), (263, 20480)])
def test_backward_many_rows(rows, cols):
    print("[case] rmsnorm_backward", rows, cols, flush=True)
    check_backward(rows_of((rows, cols), 1, BF16, 1e-3), rows_of((rows, cols), 2, BF16), torch.ones(cols, dtype=BF16),
                   rows_of((rows, cols), 3, BF16, 1e-3))


def test_backward_in_place_strides_and_no_rows():
    w = torch.ones(256, dtype=BF16)
    dy, h, dh = (rows_of((21, 256), i, BF16) for i in (1, 2, 3))
    want = check_backward(dy, h, w, dh)
    buf = dh.to(DEV)
    got = check_backward(dy, h, w, dh, dev=(dy.to(DEV), h.to(DEV), w.to(DEV), buf), dx=buf)
    assert got[0] is buf and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    buf = dy.to(DEV)
    got = check_backward(dy, h, w, dh, dev=(buf, h.to(DEV), w.to(DEV), dh.to(DEV)), dx=buf)
    assert torch.equal(got[0], want[0])
    wide = torch.zeros(21, 777, dtype=BF16, device=DEV)
    for lo in (8, 3):
        v = wide[:, lo: lo + 256]
        v.copy_(dy)
        got = check_backward(dy, h, w, dh, dev=(v, h.to(DEV), w.to(DEV), dh.to(DEV)))
        assert torch.equal(got[0], want[0])
    with pytest.raises(ValueError, match="aligned rows"):
        fgb().rmsnorm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), torch.ones(21, device=DEV), dx=wide[:, 3:259])
    dx, dw = fgb().rmsnorm_backward(torch.empty(0, 256, device=DEV), torch.empty(0, 256, device=DEV),
                                    torch.ones(256, device=DEV), torch.empty(0, device=DEV))
    assert dx.shape == (0, 256) and not dw.any()


def test_backward_is_the_forward_s_difference():
    """Through the kernels themselves, in FP32 with steps of 2^-6: the third-order error of a central difference and
    the roundings of y (38 u over the step) together stay below 2e-3 of the largest term here."""
    rows, cols, step = 2, 64, 2.0 ** -6
    g = torch.Generator().manual_seed(0)
    x, dy = torch.randn(rows, cols, generator=g), torch.randn(rows, cols, generator=g)
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    f = lambda v: (fgb().rmsnorm_quant(v.to(DEV), w.to(DEV), quant=False, y_dtype=F32)[2].cpu().double() * dy).sum(1)  # noqa: E731
    rstd = fgb().rmsnorm_quant(x.to(DEV), w.to(DEV), quant=False, y_dtype=F32)[4]
    dx, _ = fgb().rmsnorm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), rstd)
    for c in range(cols):
        e = torch.zeros(cols)
        e[c] = step
        d = (f(x + e) - f(x - e)) / (2 * step)
        assert (d - dx[:, c].cpu().double()).abs().max() < 2e-3 * float(dx.abs().max())


def test_rows_past_two_to_the_31_elements():
    """Rows whose offsets pass 2^31 elements and 2^32 bytes: the last ones as if alone, the scales among them."""
    cols, rows = 7168, 330000
    assert rows * cols > 2 ** 31
    x = torch.empty(rows, cols, dtype=BF16, device=DEV)
    x[: 1000].copy_(rows_of((1000, cols), 9, BF16))
    for lo in range(1000, rows, 1000):
        x[lo: lo + 1000].copy_(x[:1000])
    w = torch.ones(cols, dtype=BF16, device=DEV)
    q, s, y, h, rstd = fgb().rmsnorm_quant(x, w)
    last = fgb().rmsnorm_quant(x[-1000:], w)
    assert torch.equal(q[-1000:], last[0]) and torch.equal(s[-1000:], last[1]) and torch.equal(rstd[-1000:], last[4])
    dx, dw = fgb().rmsnorm_backward(x, x, w, rstd)
    one, _ = fgb().rmsnorm_backward(x[-1000:], x[-1000:], w, rstd[-1000:])
    assert torch.equal(dx[-1000:], one)


@pytest.mark.parametrize("cols", [512, 7168, 16384, 20480])
def test_backward_in_place_over_every_width(cols):
    """dx over dy and over dh, more rows than parts."""
    rows = 2100 if cols <= 2048 else 530
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(BF16).to(DEV)
    dy, h, dh = (rows_of((rows, cols), i, BF16).to(DEV) for i in (1, 2, 3))
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    want = fgb().rmsnorm_backward(dy, h, w, rstd, dh=dh)
    for k in range(2):
        t = [dy.clone(), h, dh.clone()]
        got = fgb().rmsnorm_backward(t[0], t[1], w, rstd, dh=t[2], dx=t[2 * k])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_usual_tensors():
    """What the binding's helper says of tensors, and that it leaves everything else to the checks."""
    usual = fgb()._tensors.usual
    x, w = torch.zeros(4, 96, device=DEV, dtype=BF16), torch.zeros(97, device=DEV)
    r = torch.zeros(4, 96, device=DEV)
    assert usual(x, w[:96], r, None) == (4, 96, x.data_ptr(), 1, w.data_ptr(), 0, r.data_ptr(), 0, 0, 0)
    wide = torch.zeros(4, 104, device=DEV)
    for bad in ((x, w), (x, w[1:]), (x, w[:96], wide[:, :96]), (x, w[:96], r.t()), (x, w[:96], r.half()), (x, w[:96], r[0]),
                (x[:, 1:], w[:95]), (x, w[:96], r.cpu()), (x, r), (r[0], w[:96]), (x, w[:96], 3), (x, None)):
        assert usual(*bad) is None
    with pytest.raises(ValueError, match="dh"):
        fgb().rmsnorm_backward(x, r, w[:96], torch.ones(4, device=DEV), dh=x)
    with pytest.raises(ValueError, match="same GPU|on the GPU"):
        fgb().rmsnorm_backward(x, r, w[:96], torch.ones(4))
    with pytest.raises(ValueError, match="on the GPU"):
        fgb().rmsnorm_quant(x, w[:96], residual=r, group=32, h=r.cpu())
    with pytest.raises(ValueError, match="must have shape"):
        fgb().rmsnorm_quant(x, w[:96], residual=r[:3], group=32)
    with pytest.raises(ValueError, match="weight"):
        fgb().rmsnorm_quant(x, w, group=32)
