"""The routers' workspaces on the GPU: each entry point with exactly its own, one sized for the largest batch used for
smaller ones, and the plain router's for a choice by groups."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def inputs(T, E):
    g = torch.Generator().manual_seed(T + E)
    return torch.randn(T, E, generator=g).to(DEV), (0.1 * torch.randn(E, generator=g)).to(DEV)


def space(n, fill=0xA5):
    return torch.full((n,), fill, dtype=torch.uint8, device=DEV)


def plain_need(T, E):
    """The plain router's own: 256 / lanes tokens a workgroup, 768 of them at most."""
    lanes = 8 if E <= 128 else 16 if E <= 256 else 32 if E <= 512 else 64
    blocks = max(1, min(768, -(-T * lanes // 256)))
    parts = 1 if E <= 32 else (E + 15) // 16
    return 0 if blocks == 1 else (parts + 1) * 8 + blocks * (2 * E + 1) * 4


@pytest.mark.parametrize("T,E", [(1000, 256), (1500, 256), (64, 8), (300, 64), (900, 384), (700, 1024), (20000, 256)])
def test_the_plain_router_takes_its_own_need(T, E):
    """E = 256, T = 1000: 129412 bytes."""
    z, _ = inputs(T, E)
    n = plain_need(T, E)
    assert T != 1000 or n == 129412
    how = dict(renorm=True, loss_coef=0.01)
    want = fgb().moe_router(z, 6, **how)
    buf = space(n + 64)
    got = fgb().moe_router(z, 6, workspace=buf[:n], **how)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and (buf[n:] == 0xA5).all()


@pytest.mark.parametrize("E", [8, 64, 256, 384, 1024])
def test_one_workspace_for_the_largest_batch(E):
    f = fgb()
    sizes = (5000, 1500, 1000, 513, 512, 100, 33, 2)
    for grouped in (False, True):
        size = f.moe_router_grouped_workspace_size if grouped else f.moe_router_workspace_size
        ws = space(size(sizes[0], E) + 64)
        for T in sizes:
            z, b = inputs(T, E)
            how = dict(renorm=True, loss_coef=0.01, **(dict(bias=b, groups=4, topk_groups=2) if grouped else {}))
            want = f.moe_router(z, 4, **how)
            got = f.moe_router(z, 4, workspace=ws[:-64], **how)
            assert all(torch.equal(p, q) for p, q in zip(want, got)), (T, grouped)
        assert (ws[-64:] == 0xA5).all()


@pytest.mark.parametrize("T,E", [(1000, 256), (203, 32), (40, 64), (600, 384), (5000, 64)])
def test_groups_in_the_plain_router_s_workspace(T, E):
    """Fewer workgroups: the same experts, weights and counts; the loss to a rounding of its other order."""
    f = fgb()
    z, b = inputs(T, E)
    n = f.moe_router_workspace_size(T, E)
    buf = space(n + 64)
    how = dict(score=f.ROUTER_SIGMOID, renorm=True, scale=2.5, loss_coef=0.01, bias=b, groups=8, topk_groups=3)
    want = f.moe_router(z, 3, **how)
    got = f.moe_router(z, 3, workspace=buf[:n], **how)
    assert torch.equal(want[0], got[0]) and torch.equal(want[2], got[2])
    # a weight is at most three roundings and two sums of three, in any order, from its value
    assert ((want[1] - got[1]).abs() <= 16 * 2.0 ** -24 * want[1].abs()).all()
    # each sum of p over a workgroup's tokens is within its length in roundings: T in all
    assert abs(float(want[3]) - float(got[3])) <= (T + 64) * 2.0 ** -24 * float(want[3])
    assert (buf[n:] == 0xA5).all()
    with pytest.raises(RuntimeError, match="workspace"):
        f.moe_router(z, 3, workspace=buf[: n - 1], **how)
