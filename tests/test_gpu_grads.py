"""The global gradient norm and clipping on the GPU against 64 bits.

Squares and sums are FP64: n values sum to within (n + 2) 2^-53, so sumsq is within 1e-12 of exact here, the norm
within 2^-24 more.  The factor is rounded to FP32 (2^-24) and the product to the output's type: an output is within
(2^-24 + half a step) of its value, and half the smallest subnormal where it is one."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def exact_norm(grads):
    return math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))


def check(grads, max_norm, scale=1.0, out_types=None, in_place=False):
    """grads: GPU tensors."""
    before = [g.clone() for g in grads]
    n = exact_norm(before)
    outs = None if in_place else [torch.full(g.shape, 7.0, dtype=t, device=DEV) for g, t in zip(grads, out_types)]
    norm = fgb().grad_clip(grads, max_norm, scale=scale, out=outs)
    assert norm.dtype == F32 and abs(float(norm) - scale * n) <= (2.0 ** -24 + 1e-12) * scale * n + 2.0 ** -150
    f = scale * (min(1.0, max_norm / (scale * n)) if n else 1.0)
    for i, (g, o) in enumerate(zip(before, grads if in_place else outs)):
        want = g.double() * f
        lim = (2.0 ** -24 + 1e-12 + torch.finfo(o.dtype).eps / 2 * 1.01) * want.abs()
        lim = lim + (2.0 ** -134 if o.dtype == BF16 else 2.0 ** -150)
        assert ((o.double() - want).abs() <= lim).all(), i
        if not in_place:
            assert torch.equal(grads[i], g), i
    return norm


def make(sizes, types, seed, std=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * std).to(t).to(DEV) for s, t in zip(sizes, types)]


SIZES = [1, 2, 7, 8, 9, 0, 15, 255, 2048, 2055, 16383, 16384, 16385, 0, 40000, 100003]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("clipped", [True, False])
def test_sizes_and_types(kind, clipped):
    types = [F32 if kind == "f32" or (kind == "mixed" and i % 2) else BF16 for i in range(len(SIZES))]
    grads = make(SIZES, types, 1)
    most = exact_norm(grads) * (0.3 if clipped else 3.0)
    for outs in (types, [F32] * len(types), [BF16] * len(types)):
        check(grads, most, 1.0, outs)
    check(grads, most, 0.125, types)
    check(grads, most, in_place=True)


@pytest.mark.parametrize("n", [1, 63, 64, 65, 119, 120, 121, 165, 166, 167, 240, 241, 332, 333, 500])
def test_many_tensors(n):
    print("[case] tensors", n, flush=True)
    rng = np.random.default_rng(n)
    sizes = [int(v) for v in rng.integers(0, 3000, n)]
    sizes[0] = 5
    types = [F32 if v else BF16 for v in rng.integers(0, 2, n)]
    grads = make(sizes, types, n)
    check(grads, 0.5, 1.0, types[::-1])
    check(grads, 0.5, in_place=True)


def test_views_that_start_anywhere():
    """Slices of a bucket at odd elements, in order and in place; what lies between them stays."""
    for t in (F32, BF16):
        bucket = make([70000], [t], 3)[0]
        keep = bucket.clone()
        spans = [(1, 4), (5, 1000), (1007, 17411), (20001, 20002), (20005, 69999)]
        grads = [bucket[a:b] for a, b in spans]
        check(grads, 0.1, in_place=True)
        inside = torch.zeros(70000, dtype=torch.bool, device=DEV)
        for a, b in spans:
            inside[a:b] = True
        assert torch.equal(bucket[~inside], keep[~inside])
        outs = torch.zeros(70001, dtype=BF16, device=DEV)
        g = [keep[a:b] for a, b in spans]
        fgb().grad_clip(g, 1e9, out=[outs[a + 1: b + 1] for a, b in spans])
        want = torch.zeros_like(outs)
        want[1:][inside] = keep[inside].bfloat16()
        assert torch.equal(outs, want)


def test_shapes_and_a_transposed_matrix():
    g = make([12 * 50], [F32], 4)[0].view(12, 50)
    check([g, g[3:5].clone().view(2, 1, 50)], 0.01, 1.0, [F32, BF16])
    with pytest.raises(ValueError, match="contiguous"):
        fgb().grad_clip([g.t()], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        fgb().grad_sumsq([g, g[:, :3]])
    with pytest.raises(ValueError, match="elements"):
        fgb().grad_clip([g], 1.0, out=[g[:3].clone()])
    with pytest.raises(ValueError, match="hold 1 tensors"):
        fgb().grad_clip([g], 1.0, out=[])
    for out in ([g, g], [g[0:6], g[5:11]]):
        with pytest.raises(RuntimeError, match="lies over"):
            fgb().grad_clip([o.clone() for o in out], 1.0, out=out)


def test_range_of_squares():
    """Squares far outside FP32's range, in both directions."""
    for v in (1e30, 1e-30, 3e38, 1e-44):
        for t in (F32, BF16):
            g = torch.full((3000,), v, dtype=t, device=DEV)
            n = float(g[0].double()) * math.sqrt(3000)
            s = fgb().grad_sumsq([g])
            assert abs(math.sqrt(float(s)) - n) <= 1e-12 * n
            if 0 < n < 3e38:
                check([g], n / 4, 1.0, [t])


def test_zeros_and_empty_lists():
    g = [torch.zeros(100, device=DEV), torch.empty(0, device=DEV)]
    assert float(check(g, 1.0, 1.0, [F32, BF16])) == 0
    e = [torch.empty(0, device=DEV), torch.empty(0, 5, dtype=BF16, device=DEV)]
    assert float(fgb().grad_clip(e, 1.0)) == 0 and float(fgb().grad_sumsq(e)) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(bad):
    g = make([5000, 77], [F32, BF16], 6)
    g[1][70] = bad
    out = [torch.empty_like(v) for v in g]
    norm = fgb().grad_clip(g, 0.01, scale=0.5, out=out)
    assert not math.isfinite(float(norm)) and math.isnan(float(norm)) == math.isnan(bad)
    for a, b in zip(g, out):
        assert torch.equal((a.float() * 0.5).to(a.dtype).nan_to_num(), b.nan_to_num())


def test_sumsq_adds_up_over_lists():
    a, b = make([1000, 33], [F32, BF16], 7), make([20000], [F32], 8)
    s = fgb().grad_sumsq(a)
    assert fgb().grad_sumsq(b, out=s, accumulate=True) is s
    n = exact_norm(a + b)
    assert abs(math.sqrt(float(s)) - n) <= 1e-12 * n
    norm = fgb().grad_clip(a, n / 2, sumsq=s)  # both lists' norm clips the first
    assert abs(float(norm) - n) <= 2.0 ** -23 * n
    before = make([1000, 33], [F32, BF16], 7)
    for x, y in zip(a, before):
        assert ((x.double() - y.double() / 2).abs() <= (2.0 ** -24 + 1e-12 + torch.finfo(x.dtype).eps / 2) * y.double().abs()).all()
    with pytest.raises(ValueError, match="accumulate"):
        fgb().grad_sumsq(a, accumulate=True)
    with pytest.raises(ValueError, match="sumsq"):
        fgb().grad_clip(a, 1.0, sumsq=s.float())


def test_below_the_limit_nothing_moves():
    g = make([5000, 9], [F32, BF16], 9)
    before = [v.clone() for v in g]
    fgb().grad_clip(g, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(g, before))


def test_two_runs_are_equal_bit_for_bit():
    g = make([3000000, 17, 250000], [F32, BF16, BF16], 10)
    a, b = fgb().grad_sumsq(g), fgb().grad_sumsq(g)
    assert torch.equal(a, b)


def test_past_four_gib():
    """One gradient of 2^31 + 5 elements: the last ones are counted and clipped."""
    n = 2 ** 31 + 5
    g = torch.zeros(n, dtype=BF16, device=DEV)
    g[-3:] = 2.0
    g[0] = 2.0
    norm = fgb().grad_clip([g], 1.0)
    assert float(norm) == 4.0
    assert g[-3:].tolist() == [0.5] * 3 and float(g[0]) == 0.5 and float(g[1]) == 0 and float(g[-4]) == 0


@pytest.mark.parametrize("chunks", [1, 255, 256, 257, 2047, 2049])
def test_norm_is_the_sumsq_s(chunks):
    """The norm that clipping forms itself and the one from grad_sumsq's result, bit for bit, few parts and many."""
    g = make([chunks * 8192 - 5, 3], [BF16, F32], chunks)
    outs = [torch.empty_like(v) for v in g]
    a = fgb().grad_clip(g, 0.5, out=outs)
    b = fgb().grad_clip(g, 0.5, out=[torch.empty_like(v) for v in g], sumsq=fgb().grad_sumsq(g))
    assert torch.equal(a, b)


@pytest.mark.parametrize("sizes", [[1] * 166 + [0] * 3, [0] * 3 + [1] * 166, [0] * 170 + [4] + [0] * 170, [9] * 332 + [0]])
def test_empty_tensors_around_a_full_list(sizes):
    grads = make(sizes, [F32 if i % 3 else BF16 for i in range(len(sizes))], 11)
    check(grads, 1e-3, in_place=True)
