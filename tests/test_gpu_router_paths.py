"""Router paths that depend on the numbers of tokens and choices: more tokens than the grid has lanes for (sums over
several tokens a lane, several rounds of partial results), and more slots than the experts' own lanes (9 to 32 of
few experts), ties among them."""
import numpy as np
import pytest
import torch

from oracle import router as R
from test_gpu_router import U, check, fgb

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(40000, 32, 4), (33001, 40, 5), (30011, 200, 6), (20001, 300, 8), (9001, 1024, 8)])
def test_loss_of_many_tokens(T, E, k, dtype, score):
    """The loss against 64 bits.  A lane adds up to 4 tokens' scores, a workgroup up to 32 lanes', all positive; with
    the router tests' bound of a score, (r + 28) u, the relative error is at most (r + 28 + 36) u, and more than half
    as much again is allowed for what those leave out."""
    print("[case] loss", T, E, k, dtype, score, flush=True)
    g = torch.Generator(device=DEV).manual_seed(T)
    z = (torch.randn((T, E), generator=g, device=DEV) * 1.5 + torch.randn((1, E), generator=g, device=DEV)).to(dtype)
    mask = torch.rand((T,), generator=g, device=DEV) < 0.9
    idx, w, counts, loss = fgb().moe_router(z, k, score=score, loss_coef=0.3, token_mask=mask)
    on = z.double()[mask]
    order = torch.sort(on, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(idx[mask].long(), order) and bool((idx[~mask] == -1).all())
    s = torch.softmax(on, 1) if score == R.SOFTMAX else torch.sigmoid(on)
    p = s / s.sum(1, keepdim=True)
    n = int(mask.sum())
    c = torch.bincount(order.reshape(-1), minlength=E)
    assert torch.equal(counts.long(), torch.cat([c, torch.tensor([n], device=DEV)]))
    want = 0.3 * E / (k * n * n) * float((c.double() * p.sum(0)).sum())
    r = float(on.max() - on.min())
    assert abs(float(loss) - want) <= 1.5 * (r + 28 + 43) * U * want


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(37, 40, 9), (37, 40, 12), (37, 64, 16), (37, 33, 17), (37, 100, 20), (37, 128, 32),
                                   (37, 32, 32), (37, 200, 24), (37, 300, 40), (37, 90, 33)])
def test_many_choices_of_few_experts(T, E, k, dtype, ties):
    print("[case] choices", T, E, k, dtype, ties, flush=True)
    z = torch.randn((T, E), generator=torch.Generator().manual_seed(E + k)) * 1.5
    if ties:
        z = torch.round(z * 2) / 2  # about a dozen values
        z[3:6, : E // 2] = -float("inf")  # fewer experts than slots
    z = z.to(dtype)
    check(z, k, R.SOFTMAX, True)
    check(z, k, R.SIGMOID, False)


def test_rows_of_nothing_but_nan():
    """A logit above -inf makes a token live, and NaN is not above it: a row of NaN and -inf is like one of -inf."""
    z = torch.randn((5, 20), generator=torch.Generator().manual_seed(1))
    gone = z.clone()
    gone[1], gone[3] = -float("inf"), -float("inf")
    z[1], z[3] = float("nan"), -float("inf")
    z[3, 4:9] = float("nan")
    for score in (R.SOFTMAX, R.SIGMOID):
        got, want = (fgb().moe_router(t.to(DEV), 3, score=score, loss_coef=0.5) for t in (z, gone))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert got[0][1].tolist() == [-1, -1, -1] and int(got[2][20]) == 3 and np.isfinite(float(got[3]))
        dz = fgb().moe_router_backward(z.to(DEV), got[0], got[2], torch.ones((5, 3), device=DEV),
                                       torch.ones((), device=DEV), score=score, loss_coef=0.5)
        assert bool((dz[[1, 3]] == 0).all()) and bool(torch.isfinite(dz).all())
