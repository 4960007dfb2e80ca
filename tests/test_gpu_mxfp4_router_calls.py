"""Calls of the MXFP4 and router entry points that differ from the usual in how their tensors lie in memory or in
how many there are: the same results as the usual calls, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def randn(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def equal(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


def single_row(x):
    """x [1, n] as the transpose of a column: torch calls it contiguous and its strides are (1, 1)."""
    t = x.t().clone(memory_format=torch.contiguous_format).t()
    assert t.stride() == (1, 1) and t.is_contiguous() and torch.equal(t, x)
    return t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_single_row_of_any_row_stride(dtype):
    m = fgb()
    z = randn(1, 40, dtype=dtype)
    for lg in (single_row(z), torch.cat([z] * 3, 1)[:, 40:80]):
        want, got = (m.moe_router(t, 4, renorm=True, loss_coef=0.1) for t in (z, lg))
        assert equal(want, got)
        w = torch.ones((1, 4), device=DEV)
        assert torch.equal(m.moe_router_backward(z, want[0], want[2], w), m.moe_router_backward(lg, got[0], got[2], w))
    x = randn(1, 96, seed=1, dtype=dtype)
    stacked = torch.empty_strided((3, 1, 96), (96, 1, 1), dtype=dtype, device=DEV)
    stacked.copy_(randn(3, 1, 96, seed=2, dtype=dtype))
    apart = randn(3, 2, 96, seed=3, dtype=dtype)[:, :1]
    for quant in (m.mxfp4_quant, m.mxfp4_quant_t):
        assert equal(quant(x), quant(single_row(x)))
        assert equal(quant(stacked.clone(memory_format=torch.contiguous_format)), quant(stacked))
        assert equal(quant(apart.contiguous()), quant(apart))
    empty = torch.empty((40, 0), dtype=dtype, device=DEV).t()
    assert m.moe_router(empty, 4)[0].shape == (0, 4)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_a_single_row_in_a_product(fmt):
    m = fgb()
    x, (b, sb) = randn(1, 256), m.mxfp4_quant(randn(16, 256, seed=1))
    a, sa = m.mxfp4_quant(x) if fmt == "e2m1" else m.fp8_quant_rowwise(x)
    f = m.E2M1 if fmt == "e2m1" else m.E4M3
    want = m.mxfp4_gemm(a, sa, b, sb, a_fmt=f)
    d = single_row(torch.zeros_like(want))
    assert m.mxfp4_gemm(single_row(a), sa, b, sb, a_fmt=f, d=d) is d
    assert torch.equal(want, d)


def test_a_single_row_in_the_fp8_calls():
    m = fgb()
    x, w = randn(1, 256), randn(128, 256, seed=1)
    xq, xs = m.fp8_quant_rowwise(x)
    assert equal((xq, xs), m.fp8_quant_rowwise(single_row(x)))
    wq, ws = m.fp8_quant_blockwise(w)
    assert torch.equal(m.fp8_block_gemm(xq, xs, m.ROW1x128, wq, ws, m.BLOCK128),
                       m.fp8_block_gemm(single_row(xq), xs, m.ROW1x128, wq, ws, m.BLOCK128))


def test_slices_of_stacked_scales():
    """Scales of 5 rows and one step take 40 bytes: the odd slices of a stack start at a multiple of 8 only."""
    m = fgb()
    q, s = m.mxfp4_quant(randn(4, 5, 160))
    xq, xs = m.mxfp4_quant(randn(4, 5, 160, seed=1))
    x8, x8s = m.fp8_quant_rowwise(randn(5, 256, seed=2))
    w8, w8s = m.mxfp4_quant(randn(4, 5, 256, seed=3))
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    for i in range(4):
        assert s[i].data_ptr() % 16 == 8 * (i % 2) and s[i].is_contiguous()
        whole = [t[i].clone() for t in (q, s, xq, xs, w8, w8s)]
        assert torch.equal(m.mxfp4_dequant(q[i], s[i]), m.mxfp4_dequant(*whole[:2]))
        assert torch.equal(m.mxfp4_gemm(xq[i], xs[i], q[i], s[i]), m.mxfp4_gemm(*whole[2:4], *whole[:2]))
        assert torch.equal(m.mxfp4_gemm(x8, x8s, w8[i], w8s[i], a_fmt=m.E4M3),
                           m.mxfp4_gemm(x8, x8s, *whole[4:], a_fmt=m.E4M3))
    got = m.mxfp4_grouped_gemm(xq[1], xs[1], q[1:3], s[1:3], off, a_fmt=m.E2M1)
    want = m.mxfp4_grouped_gemm(xq[1].clone(), xs[1].clone(), q[1:3].clone(), s[1:3].clone(), off, a_fmt=m.E2M1)
    assert torch.equal(got, want)


def test_more_tiles_than_one_launch_holds():
    """2^24 workgroups of 256 threads are more than a launch takes: many short matrices, and 2^35 values back."""
    m = fgb()
    G = (1 << 24) + 5
    x = torch.empty((G, 1, 32), dtype=torch.bfloat16, device=DEV).normal_()
    q, s = m.mxfp4_quant(x)
    flat, fs = m.mxfp4_quant(x.view(G, 32))  # rows of one matrix: 32 to a workgroup
    assert torch.equal(q.view(G, 16), flat)
    assert torch.equal(s.view(G, 8), fs.view(G, 8))
    del x, q, s, flat, fs
    rows, cols = (1 << 22) + 3, 8192
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV).random_()
    s = torch.empty((cols // 256, rows, 8), dtype=torch.uint8, device=DEV).random_(120, 135)
    d = m.mxfp4_dequant(q, s, out_dtype=torch.bfloat16)
    for r in (slice(0, 3), slice((1 << 22) - 2, rows)):
        assert torch.equal(d[r], m.mxfp4_dequant(q[r].contiguous(), s[:, r].contiguous(), out_dtype=torch.bfloat16))


@pytest.mark.parametrize("M", [1, 3])
def test_accumulating_needs_a_sum_to_add_to(M):
    m = fgb()
    a, sa = m.mxfp4_quant(randn(M, 256))
    b, sb = m.mxfp4_quant(randn(16, 256, seed=1))
    with pytest.raises(ValueError, match="accumulate needs d"):
        m.mxfp4_gemm(a, sa, b, sb, out_dtype=torch.float32, accumulate=True)
    d = torch.ones((M, 16), device=DEV)
    m.mxfp4_gemm(a, sa, b, sb, d=d, accumulate=True)
    assert torch.equal(d, 1 + m.mxfp4_gemm(a, sa, b, sb, out_dtype=torch.float32))


def test_more_moss_groups_than_one_launch_holds():
    m = fgb()
    x = torch.empty(((1 << 16) + 1, 8192), dtype=torch.bfloat16, device=DEV).normal_()
    q, s2, s1 = m.mx2_quant(x, g1=32)  # 256 groups a row
    for r in (slice(0, 2), slice((1 << 15) - 1, (1 << 15) + 1), slice((1 << 16) - 1, (1 << 16) + 1)):
        assert equal((q[r], s2[r], s1[r]), m.mx2_quant(x[r].contiguous(), g1=32))


def test_more_tokens_than_one_launch_permutes():
    m = fgb()
    T, G, H = (1 << 26) + 5, 4, 128
    xq = torch.empty((T, H), dtype=torch.uint8, device=DEV).random_()
    xs = torch.empty((T, 1), dtype=torch.uint8, device=DEV).random_()
    idx = torch.empty((T, 1), dtype=torch.int32, device=DEV).random_(0, G)
    q, s, row_map, offs = m.permute_pad(xq, xs, idx, G)
    at = row_map[:, 0].long()
    for lo in range(0, T, 1 << 24):
        part = slice(lo, lo + (1 << 24))
        assert torch.equal(q[at[part]], xq[part]) and torch.equal(s[at[part]], xs[part])
    counts, off = torch.bincount(idx[:, 0], minlength=G).tolist(), offs.tolist()
    for g in range(G):
        assert bool((q[off[g] + counts[g]:off[g + 1]] == 0).all())
