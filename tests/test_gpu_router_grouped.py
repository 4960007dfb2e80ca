"""The router whose choice a bias and groups decide, on the GPU against the 64-bit reference.  Ids and counts are
exact: both sides compare FP32(FP32(s) + bias), and a score in 64 bits is rounded to another FP32 number by one side
only if it lies within 2^-52 of a border.  Weights, loss and gradients hold the bounds of test_gpu_router.py, r being
the range of the logits."""
import numpy as np
import pytest
import torch

from oracle import router as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def logits(T, E, seed, dtype=F32, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * scale).to(dtype)


def biases(E, seed, scale=0.1):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed)) * scale


def check(z, k, bias, groups, kg, score, renorm, scale=1.0, coef=0.01, mask=None, seed=0, view=None, reach=None):
    """Forward and backward; reach: the range of the logits that matter, where it is not that of all of them."""
    T, E = z.shape
    zd = z.to(DEV) if view is None else view
    zn = z.double().numpy()
    bn = None if bias is None else bias.numpy()
    m = None if mask is None else torch.as_tensor(mask)
    idx0 = R.choose(zn, k, score, bn, groups, kg, mask)
    f = R.forward(zn, k, score, renorm, scale, coef, mask, idx=idx0)
    idx, w, counts, loss = fgb().moe_router(
        zd, k, score=score, renorm=renorm, scale=scale, loss_coef=coef, token_mask=None if m is None else m.to(DEV),
        bias=None if bias is None else bias.to(DEV), groups=groups, topk_groups=kg)
    assert np.array_equal(idx.cpu().numpy(), f["idx"])
    assert np.array_equal(counts.cpu().numpy(), f["counts"])
    fin = zn[np.isfinite(zn)]
    r = reach if reach is not None else float(fin.max() - fin.min()) if fin.size else 0.0
    tol = (r + 28) * U
    w = w.double().cpu().numpy()
    assert (np.abs(w - f["weights"]) <= 4 * tol * np.abs(f["weights"]) + 1e-37).all()
    if coef:
        # a p below FP32's smallest number is off by at most 2^-150: in coef E / (k n^2) sum counts_e sum_t p, where
        # the counts sum to at most k n, that comes to coef E 2^-150; the loss's own rounding to 2^-150 more
        assert abs(float(loss) - f["loss"]) <= 4 * tol * abs(f["loss"]) + (abs(coef) * E + 1) * 2.0 ** -150
    rng = np.random.default_rng(seed)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    want = R.backward(zn, f["idx"], f["counts"], dw, 0.7, score, renorm, scale, coef)
    got = fgb().moe_router_backward(zd, idx, counts, torch.from_numpy(dw).to(DEV), torch.tensor(0.7, device=DEV),
                                    score=score, renorm=renorm, scale=scale, loss_coef=coef)
    n = max(int(f["counts"][E]), 1)
    big = 0.7 * coef * E / (k * n * n) * f["counts"][:E].max(initial=0) + scale * np.abs(dw).max(initial=0.0)
    lim = 16 * tol * big + 1e-37
    if z.dtype == BF16:
        lim = lim + 2.0 ** -8 * (np.abs(want) + lim) + 2.0 ** -134
    assert (np.abs(got.double().cpu().numpy() - want) <= lim).all()
    return f


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k,G,kg", [
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 8, 4, 8, 4), (5, 64, 6, 8, 3), (33, 160, 6, 8, 3), (40, 96, 5, 3, 1),
    (17, 21, 4, 7, 5), (9, 64, 64, 64, 64), (70, 128, 8, 16, 2), (19, 512, 8, 64, 9), (7, 1024, 10, 32, 5),
    (11, 1020, 64, 4, 1), (21, 260, 8, 2, 1), (6, 384, 8, 1, 1), (700, 40, 5, 10, 3), (13, 63, 20, 9, 9),
])
def test_grouped(T, E, k, G, kg, dtype, biased, score):
    if G == 1 and not biased:
        biased = True  # (the plain router)
    print("[case] grouped", T, E, k, G, kg, dtype, biased, score, flush=True)
    for renorm in (False, True):
        check(logits(T, E, T + E, dtype), k, biases(E, E) if biased else None, G, kg, score, renorm,
              scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,G,kg", [(24, 4, 2), (100, 20, 6), (300, 3, 2)])
def test_masks(E, G, kg, biased, score):
    """Disabled experts, whole groups of them, rows with nothing left, padding tokens, NaN in an unlive row."""
    print("[case] masks", E, G, kg, biased, score, flush=True)
    T, S = 97, E // G
    z = logits(T, E, 3)
    g = torch.Generator().manual_seed(4)
    z[torch.rand((T, E), generator=g) < 0.3] = -np.inf
    z[:, :S] = -np.inf                          # group 0 has nothing
    z[5:20, : (G - 1) * S] = -np.inf            # only the last group has
    z[5:20, (G - 1) * S + 1:] = -np.inf         # ... and there one expert at most
    z[30] = -np.inf
    z[31] = -np.inf
    z[31, 3] = float("nan")
    mask = (torch.rand(T, generator=g) < 0.8).numpy()
    z[40:44] = torch.finfo(F32).min             # the lowest finite value is a value
    mask[40:44] = True
    usual = z[torch.isfinite(z) & (z > -1e30)]
    for renorm in (False, True):
        f = check(z, 4, biases(E, 1) if biased else None, G, kg, score, renorm, mask=mask,
                  reach=float(usual.max() - usual.min()))
        assert (f["idx"][30] == -1).all() and (f["idx"][31] == -1).all()


def test_ties_go_to_the_lowest():
    z = torch.zeros(5, 32)
    z[1, 16:] = 1.0
    z[2, [3, 11, 19, 27]] = 2.0
    z[3, ::2] = -0.0
    for bias in (None, torch.zeros(32), torch.full((32,), 0.25)):
        f = check(z, 6, bias, 4, 2, R.SIGMOID, True)
        assert f["idx"][0].tolist() == [0, 1, 2, 3, 4, 5]


def test_saturated_scores_tie_under_a_bias():
    """Logits of 20 and more all have the score 1: the bias, then the id, decides."""
    z = torch.linspace(20, 60, 16).repeat(3, 1)
    b = torch.zeros(16)
    b[[5, 9]] = 1e-3
    f = check(z, 4, b, 2, 2, R.SIGMOID, True)
    assert f["idx"][0].tolist() == [5, 9, 0, 1]


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_chosen_far_below_the_largest(score, dtype):
    """A bias, or groups, choose experts whose scores vanish beside the largest: renormed weights and their gradients
    stay finite and right.  r is the range of the chosen logits and of exp's arguments: at most 400."""
    E = 32
    z = logits(9, E, 1, dtype, 0.5)
    z[:, :8] += 100
    z[3:, 8:16] -= 250
    b = torch.zeros(E)
    b[8:16] = 5.0
    check(z, 4, b, 1, 1, score, True, reach=400.0)
    check(z, 4, b, 4, 1, score, True, reach=400.0)
    check(z, 4, b, 4, 2, score, False, reach=400.0)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_bias_of_infinities_and_nan(score):
    z = logits(11, 24, 2)
    b = biases(24, 2)
    b[[0, 5, 6, 7, 8, 9, 10, 11]] = -np.inf  # group 1 (of 6) is disabled
    b[13] = float("nan")
    check(z, 5, b, 4, 2, score, False)
    b[13] = np.inf
    f = check(z, 5, b, 4, 2, score, False)
    assert (f["idx"][:, 0] == 13).all()
    b[:] = -np.inf
    f = check(z, 5, b, 4, 2, score, False)
    assert (f["idx"] == -1).all() and f["counts"][24] == 0


def test_infinite_logit():
    """+inf has the score 1 (softmax: alone); it is chosen first."""
    z = logits(3, 16, 1)
    z[1, 7] = np.inf
    for score in (R.SOFTMAX, R.SIGMOID):
        idx = fgb().moe_router(z.to(DEV), 3, score=score, bias=torch.zeros(16, device=DEV), groups=4, topk_groups=2)[0]
        assert np.array_equal(idx.cpu().numpy(), R.choose(z.double().numpy(), 3, score, np.zeros(16), 4, 2))
        assert int(idx[1, 0]) == 7


def test_strided_logits_and_no_tokens():
    base = logits(50, 70, 1).to(DEV)
    for v in (base[:, 3:67], base[::3, :64], base[7:8, 1:65]):
        check(v.cpu(), 6, biases(64, 1), 8, 3, R.SIGMOID, True, view=v)
    idx, w, counts, loss = fgb().moe_router(torch.empty(0, 64, device=DEV), 6, bias=biases(64, 1).to(DEV), groups=8,
                                            topk_groups=3, loss_coef=0.1)
    assert idx.shape == (0, 6) and not counts.any() and float(loss) == 0


@pytest.mark.parametrize("T", [255, 256, 257, 5000, 30011])
def test_many_tokens(T):
    print("[case] many tokens", T, flush=True)
    check(logits(T, 64, T), 6, biases(64, 5), 8, 4, R.SIGMOID, True, scale=2.5)


def test_zero_bias_and_all_groups_is_the_plain_choice():
    z = logits(500, 128, 8).to(DEV)
    a = fgb().moe_router(z, 8, renorm=True)
    b = fgb().moe_router(z, 8, renorm=True, groups=8, topk_groups=8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("E", [1, 2, 63, 64, 65, 256, 1000, 1024])
def test_bias_update(E):
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 2 ** 31 // E if E > 1 else 100, E + 1).astype(np.int32)
    counts[: E // 3] = counts[:E].mean() if E > 2 else counts[0]
    b = biases(E, 1)
    want = b + 1e-3 * torch.from_numpy(np.sign(int(counts[:E].sum()) - counts[:E].astype(np.int64) * E)).float()
    bd, cd = b.to(DEV), torch.from_numpy(counts).to(DEV)
    assert torch.equal(fgb().moe_bias_update(bd, cd, 1e-3).cpu(), want)
    assert fgb().moe_bias_update(bd, cd, 1e-3, out=bd) is bd and torch.equal(bd.cpu(), want)


@pytest.mark.parametrize("T,E,k,G,kg", [
    (9001, 128, 8, 64, 20), (9001, 64, 8, 16, 5), (9001, 256, 8, 64, 17), (5001, 512, 8, 4, 2), (9001, 96, 4, 2, 1),
    (3, 2, 1, 2, 1), (5, 3, 2, 3, 2), (300, 3, 1, 1, 1), (9000, 9, 3, 3, 2), (4500, 768, 7, 48, 11),
])
def test_group_shapes_over_many_tokens(T, E, k, G, kg):
    """Every way a group's two largest are found, with few and many lanes a token and up to 64 groups."""
    print("[case] group shapes", T, E, k, G, kg, flush=True)
    for biased, score, dtype in ((True, R.SIGMOID, F32), (False, R.SOFTMAX, BF16), (True, R.SOFTMAX, BF16)):
        if biased or G > 1:
            check(logits(T, E, E, dtype), k, biases(E, 3) if biased else None, G, kg, score, True)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("E,k", [(432, 1), (32, 1), (100, 4), (700, 12), (64, 40)])
def test_a_lone_expert_s_weight_is_constant(E, k, score):
    """Renormed, the weight of a token's only expert is 1 whatever its logit: gradients of the weights add nothing, bit
    for bit, where one slot was filled."""
    T = 300
    z = logits(T, E, E)
    g = torch.Generator().manual_seed(5)
    only = torch.randint(0, E, (T,), generator=g)
    if k > 1:
        z[::2] = -np.inf
        z[torch.arange(0, T, 2), only[::2]] = 0.5
    zd = z.to(DEV)
    how = dict(score=score, renorm=True, scale=2.5, loss_coef=0.01)
    idx, w, counts, _ = fgb().moe_router(zd, k, bias=biases(E, 2).to(DEV), **how)
    dw = torch.randn(T, k, generator=g).to(DEV)
    one = torch.ones((), device=DEV)
    with_w = fgb().moe_router_backward(zd, idx, counts, dw, one, **how)
    without = fgb().moe_router_backward(zd, idx, counts, None, one, **how)
    rows = slice(None) if k == 1 else slice(0, None, 2)
    assert torch.equal(with_w[rows], without[rows]) and (w[rows, 0] == 2.5).all()
    if k > 1:
        assert not torch.equal(with_w[1::2], without[1::2])


def test_logits_past_two_to_the_31():
    """More than 2^31 logits: the last tokens as if alone (1024 experts have the same lanes in both calls)."""
    T, E, k = 2 ** 21 + 77, 1024, 8
    z = torch.empty(T, E, dtype=BF16, device=DEV)
    part = logits(4096, E, 1, BF16).to(DEV)
    for lo in range(0, T, 4096):
        z[lo: lo + 4096].copy_(part[: min(4096, T - lo)])
    z[-50:].copy_(logits(50, E, 2, BF16))
    how = dict(score=R.SIGMOID, renorm=True, scale=2.5, loss_coef=0.01)
    choice = dict(bias=biases(E, 1).to(DEV), groups=8, topk_groups=4)
    idx, w, counts, loss = fgb().moe_router(z, k, **how, **choice)
    one = fgb().moe_router(z[-50:], k, **how, **choice)
    assert torch.equal(idx[-50:], one[0]) and torch.equal(w[-50:], one[1])
    assert int(counts[E]) == T and int(counts[:E].sum()) == T * k and float(loss) > 0
    dw = torch.ones(T, k, device=DEV)
    dw[:, 0] = 0.5
    dz = fgb().moe_router_backward(z, idx, counts, dw, torch.ones((), device=DEV), **how)
    few = fgb().moe_router_backward(z[-50:], idx[-50:], counts, dw[-50:], torch.ones((), device=DEV), **how)
    assert torch.equal(dz[-50:], few)
