"""The MoE router on the GPU against the 64-bit reference.  Ids and counts are exact.  With u = 2^-24: a score's
relative error is at most (r + 2 + n + 4) u, r the logits' range (rounding of z - max, times exp's slope), 2 ulp for
exp, n <= 22 additions in a sum and a few operations more, so 2e-6 covers r <= 8 and (r + 28) u the rest; a
gradient is a few such terms, within 16 (r + 28) u of the largest of |g| and |D|, and half a BF16 ulp more where it
is BF16."""
import numpy as np
import pytest
import torch

from oracle import router as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def logits(T, E, seed, dtype=torch.float32, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * scale).to(dtype)


def check(z, k, score, renorm, scale=1.0, coef=0.01, mask=None, seed=0, view=None):
    """Forward and backward of z (CPU tensor); view: the GPU tensor to use in its place."""
    T, E = z.shape
    zd = z.to(DEV) if view is None else view
    zn = z.double().numpy()
    m = None if mask is None else torch.as_tensor(mask)
    f = R.forward(zn, k, score, renorm, scale, coef, mask)
    idx, w, counts, loss = fgb().moe_router(zd, k, score=score, renorm=renorm, scale=scale, loss_coef=coef,
                                            token_mask=None if m is None else m.to(DEV))
    assert np.array_equal(idx.cpu().numpy(), f["idx"])
    assert np.array_equal(counts.cpu().numpy(), f["counts"])
    fin = zn[np.isfinite(zn)]
    r = float(fin.max() - fin.min()) if fin.size else 0.0
    tol = (r + 28) * U
    w = w.double().cpu().numpy()
    assert (np.abs(w - f["weights"]) <= 4 * tol * np.abs(f["weights"]) + 1e-37).all()
    if coef:
        assert abs(float(loss) - f["loss"]) <= 4 * tol * abs(f["loss"])
    else:
        assert loss is None
    rng = np.random.default_rng(seed)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    for use_w, dl in ((True, 0.7), (True, None), (False, 1.3)):
        want = R.backward(zn, f["idx"], f["counts"], dw * use_w, dl or 0.0, score, renorm, scale, coef)
        got = fgb().moe_router_backward(
            zd, idx, counts, torch.from_numpy(dw).to(DEV) if use_w else None,
            None if dl is None else torch.tensor(dl, device=DEV), score=score, renorm=renorm, scale=scale, loss_coef=coef)
        assert got.dtype == z.dtype and got.shape == z.shape
        n = max(int(f["counts"][E]), 1)
        g = (dl or 0.0) * coef * E / (k * n * n) * (f["counts"][:E].max() if E else 0)
        big = abs(g) + use_w * scale * np.abs(dw).max(initial=0.0)
        lim = 16 * tol * big + 1e-37
        if z.dtype == torch.bfloat16:
            lim = lim + 2.0 ** -8 * (np.abs(want) + lim) + 2.0 ** -134
        assert (np.abs(got.double().cpu().numpy() - want) <= lim).all()
    return f


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 32, 8), (2, 8, 8), (3, 33, 4), (5, 64, 64), (9, 65, 6), (100, 16, 2), (70, 128, 8), (33, 130, 7),
    (41, 256, 8), (40, 257, 6), (17, 512, 10), (19, 600, 3), (11, 1024, 64), (700, 40, 5),
])
def test_router(T, E, k, dtype, renorm, score):
    print("[case] router", T, E, k, dtype, renorm, score, flush=True)
    check(logits(T, E, T + E, dtype), k, score, renorm, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [24, 100, 300])
def test_masks(E, renorm, score):
    """Padding tokens, disabled experts, tokens with fewer experts than slots and with none."""
    T, k = 60, 5
    z = logits(T, E, 4)
    g = torch.Generator().manual_seed(1)
    z[torch.rand((T, E), generator=g) < 0.3] = -float("inf")
    z[7], z[8, 3:] = -float("inf"), -float("inf")
    z[9], z[9, E - 1] = -float("inf"), 0.5
    mask = (torch.rand(T, generator=g) < 0.8).numpy()
    mask[[7, 8, 9]] = True
    f = check(z, k, score, renorm, mask=mask)
    assert (f["idx"][7] == -1).all() and (f["idx"][9] >= 0).sum() == 1
    check(z, k, score, renorm, mask=np.zeros(T, bool))  # nothing live: the loss is 0
    check(torch.full((4, E), -float("inf")), k, score, renorm)


@pytest.mark.parametrize("E", [6, 64, 200])
def test_ties_go_to_the_lowest_id(E):
    z = torch.zeros((5, E))
    z[1] = 1.0
    z[2, E // 2:] = -0.0
    z[3] = torch.randint(0, 2, (E,), generator=torch.Generator().manual_seed(2)).float()
    f = check(z, 4, R.SOFTMAX, True)
    assert f["idx"][0].tolist() == [0, 1, 2, 3] and f["idx"][2].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_far_logits(score, renorm):
    """Logits whose scores under- or overflow if formed naively; masks written as the type's lowest value."""
    z = logits(12, 40, 3)
    z[:3] -= 200.0
    z[3:6] += 200.0
    z[6:9] *= 40.0
    z[9, 5:] = torch.finfo(torch.float32).min
    z[10] = torch.finfo(torch.float32).min
    zn = z.double().numpy()
    idx, w, counts, loss = fgb().moe_router(z.to(DEV), 4, score=score, renorm=renorm, loss_coef=0.1)
    f = R.forward(zn, 4, score, renorm, 1.0, 0.1)
    assert np.array_equal(idx.cpu().numpy(), f["idx"]) and np.array_equal(counts.cpu().numpy(), f["counts"])
    tol = (400 + 28) * U  # rows differ: their own range is below 400 where scores do not vanish
    assert (np.abs(w.double().cpu().numpy() - f["weights"]) <= 4 * tol * np.abs(f["weights"]) + 1e-37).all()
    assert abs(float(loss) - f["loss"]) <= 4 * tol * f["loss"]
    dw = torch.ones((12, 4), device=DEV) * torch.arange(4, device=DEV)
    dz = fgb().moe_router_backward(z.to(DEV), idx, counts, dw, torch.ones((), device=DEV), score=score, renorm=renorm,
                                   loss_coef=0.1)
    want = R.backward(zn, f["idx"], f["counts"], dw.double().cpu().numpy(), 1.0, score, renorm, 1.0, 0.1)
    assert (np.abs(dz.double().cpu().numpy() - want) <= 16 * tol * 4).all()


def test_nan_is_not_chosen_and_not_hidden():
    z = logits(6, 20, 8)
    z[2, 4] = float("nan")
    z[4, 7] = float("inf")
    idx, w, counts, loss = fgb().moe_router(z.to(DEV), 3, loss_coef=1.0)
    idx, w = idx.cpu(), w.cpu()
    assert 4 not in idx[2].tolist() and torch.isnan(w[2]).all() and np.isnan(float(loss))
    assert idx[4, 0] == 7
    good = [0, 1, 3, 5]
    f = R.forward(z[good].double().numpy(), 3)
    assert np.array_equal(idx[good].numpy(), f["idx"]) and np.allclose(w[good].numpy(), f["weights"], rtol=4e-6, atol=0)


def test_strides_and_a_large_batch():
    wide = logits(5000, 72, 6).to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        w = wide.to(dtype)
        view = w[1::2, 3:60]
        check(view.cpu(), 6, R.SOFTMAX, True, view=view)


def test_the_gradient_against_differences():
    """The GPU's gradient against central differences of the objective in 64 bits."""
    T, E, k = 6, 10, 3
    z = logits(T, E, 12)
    dw = np.random.default_rng(3).normal(size=(T, k)).astype(np.float32)
    for score in (R.SOFTMAX, R.SIGMOID):
        for renorm in (False, True):
            idx, _, counts, _ = fgb().moe_router(z.to(DEV), k, score=score, renorm=renorm, scale=1.5, loss_coef=0.4)
            dz = fgb().moe_router_backward(z.to(DEV), idx, counts, torch.from_numpy(dw).to(DEV),
                                           torch.tensor(0.9, device=DEV), score=score, renorm=renorm, scale=1.5,
                                           loss_coef=0.4).double().cpu().numpy()
            how = (idx.cpu().numpy(), counts.cpu().numpy(), dw.astype(np.float64), 0.9, score, renorm, 1.5, 0.4)
            zn = z.double().numpy()
            for t in range(T):
                for e in range(E):
                    up, dn = zn.copy(), zn.copy()
                    up[t, e] += 1e-5
                    dn[t, e] -= 1e-5
                    want = (R.objective(up, *how) - R.objective(dn, *how)) / 2e-5
                    assert abs(want - dz[t, e]) <= 16 * 40 * U * 8 + 1e-9


def test_empty_batch_and_repeats():
    idx, w, counts, loss = fgb().moe_router(torch.empty((0, 16), device=DEV), 2, loss_coef=1.0)
    assert idx.shape == (0, 2) and bool((counts == 0).all()) and float(loss) == 0.0
    assert fgb().moe_router_backward(torch.empty((0, 16), device=DEV), idx, counts).shape == (0, 16)
    z = logits(3000, 48, 2).to(DEV)
    first = fgb().moe_router(z, 4, loss_coef=1.0)
    for _ in range(3):
        again = fgb().moe_router(z, 4, loss_coef=1.0)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
