"""MXFP4 quantisation and products on the GPU against the 64-bit reference: codes, scales and decoded values bit
for bit; products within the bound of K products summed in FP32, (K - 1) 2^-24 sum |product|, and half a BF16
ulp more where D is BF16."""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def say(*a):
    print("[case]", *a, flush=True)


def values(rows, cols, seed, dtype=torch.float32, spread=8):
    """Normal values, each row times a power of two, each group of 32 times another: the scales differ."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    x = x * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), generator=g).float())
    k = torch.exp2(torch.randint(-3, 4, (rows, (cols + 31) // 32), generator=g).float())
    return (x * k.repeat_interleave(32, 1)[:, :cols]).to(dtype)


def same(got, want):
    return np.array_equal(got.cpu().numpy(), want)


def check_product(got, av, bv, base=0.0):
    """got = av bv^T (+ base) within the bounds above; av, bv the operands' exact values."""
    ref, mag = O.gemm(av, bv)
    K = av.shape[1]
    tol = K * 2.0 ** -24 * mag + 2.0 ** -24 * (np.abs(ref) + np.abs(base)) + 1e-44
    ref = ref + base
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -134
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))


# ---- quantisation -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 288), (31, 96), (129, 256), (257, 480), (300, 1056)])
def test_quant_both_directions(rows, cols, rule, dtype):
    say("quant", rows, cols, rule, dtype)
    x = values(rows, cols, rows * 7 + cols, dtype)
    if rows > 2:
        x[1, :32] = 0.0  # an all-zero group
        x[2] = -x[2].abs()
    q, s = O.quant(x.double().numpy(), rule)
    qt, st = O.quant(x.double().t().numpy(), rule)
    a = fgb().mxfp4_quant(x.to(DEV), rule=rule)
    b = fgb().mxfp4_quant_t(x.to(DEV), rule=rule)
    assert same(a[0], q) and same(a[1], s)
    assert same(b[0], q) and same(b[1], s)
    assert same(b[2], qt) and same(b[3], st)


def test_quant_every_tie_and_edge():
    """Every E2M1 value and tie at many exponents, the largest and smallest floats, subnormals, infinities and NaN."""
    m = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    rows = []
    for e in (-149, -140, -127, -126, -125, -60, -2, 0, 1, 60, 124):
        for d in (0, 1, -1):
            with np.errstate(over="ignore"):
                v = np.ldexp(m, e).astype(np.float32)
            v = np.nextafter(v, np.float32(np.inf * d), dtype=np.float32) if d else v
            rows.append(np.concatenate([v, [0.0], -v, [-0.0]]))
    top = np.finfo(np.float32).max
    rows += [np.full(32, top), np.r_[top, np.zeros(31)], np.r_[np.inf, np.ones(31)], np.r_[np.ones(31), np.nan],
             np.r_[-np.inf, np.nan, np.zeros(30)]]
    x = np.stack(rows).astype(np.float32)
    for rule in (0, 1):
        q, s = O.quant(x, rule)
        got = fgb().mxfp4_quant(torch.from_numpy(x).to(DEV), rule=rule)
        assert same(got[1], s)
        fine = O.row_scales(s, 1)[:, 0] != 255  # a NaN group's codes mean nothing
        assert same(got[0][torch.from_numpy(fine).to(DEV)], q[fine])
        back = fgb().mxfp4_dequant(*got).cpu().numpy()
        want = O.dequant(q, s)
        assert np.isnan(back[~fine]).all() and np.array_equal(back[fine], want[fine].astype(np.float32))


def test_quant_strides_and_stacks():
    x = values(70, 512, 1, torch.bfloat16).to(DEV)
    view = x[3:60:2, 64:352]  # a row stride of 1024 elements, an offset of 128 bytes
    q, s = O.quant(view.double().cpu().numpy())
    for got in (fgb().mxfp4_quant(view), fgb().mxfp4_quant_t(view)):
        assert same(got[0], q) and same(got[1], s)
    odd = x[:, 1:289]  # rows that start at an odd element
    q, s = O.quant(odd.double().cpu().numpy())
    got = fgb().mxfp4_quant(odd)
    assert same(got[0], q) and same(got[1], s)
    w = torch.stack([values(45, 96, 10 + i, torch.float32) for i in range(3)])
    got = fgb().mxfp4_quant_t(w.to(DEV))
    alone = fgb().mxfp4_quant(w.to(DEV))
    for i in range(3):
        q, s = O.quant(w[i].double().numpy())
        qt, st = O.quant(w[i].double().t().numpy())
        assert same(got[0][i], q) and same(got[1][i], s) and same(got[2][i], qt) and same(got[3][i], st)
        assert same(alone[0][i], q) and same(alone[1][i], s)


def test_quant_empty():
    for shape in [(0, 64), (5, 0)]:
        q, s = fgb().mxfp4_quant(torch.empty(shape, device=DEV))
        assert q.numel() == 0 and s.numel() == 0
        assert fgb().mxfp4_dequant(q, s).numel() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (17, 288), (64, 2048)])
def test_dequant_every_code_and_scale(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows)
    q = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    s = torch.randint(0, 256, ((cols + 255) // 256, rows, 8), generator=g, dtype=torch.int32).to(torch.uint8)
    got = fgb().mxfp4_dequant(q.to(DEV), s.to(DEV), out_dtype=dtype).cpu()
    want = torch.from_numpy(O.dequant(q.numpy(), s.numpy())).to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


# ---- dense products ------------------------------------------------------------------------

def operand_a(M, K, fmt, seed):
    """(codes, scales) on the GPU and their exact values."""
    x = values(M, K, seed, torch.bfloat16)
    if fmt == "e2m1":
        q, s = O.quant(x.double().numpy())
        return torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), O.dequant(q, s)
    q, s = fgb().fp8_quant_rowwise(x.to(DEV))
    v = fgb().fp8_dequant(q, s, fgb().ROW1x128).double().cpu().numpy()
    return q, s, v


def operand_b(N, K, seed):
    q, s = O.quant(values(N, K, seed, spread=4).double().numpy())
    return torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), O.dequant(q, s)


FMT = {"e2m1": 2, "e4m3": 0}


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 128), (1, 2048, 1024), (2, 33, 256), (5, 130, 640), (16, 64, 128), (17, 100, 384), (33, 257, 1152),
    (64, 512, 2048), (77, 2112, 1536), (130, 96, 256), (255, 300, 512), (256, 256, 256), (300, 515, 896),
    (520, 777, 1280),
])
def test_gemm(M, N, K, fmt, out):
    say("gemm", M, N, K, fmt, out)
    a, sa, av = operand_a(M, K, fmt, M + K)
    b, sb, bv = operand_b(N, K, N)
    check_product(fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=FMT[fmt], out_dtype=out), av, bv)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("K", [32, 64, 96, 224, 288, 352, 480, 544, 992])
def test_gemm_k_that_no_step_divides(M, K):
    a, sa, av = operand_a(M, K, "e2m1", K)
    b, sb, bv = operand_b(70, K, K + 1)
    # what lies behind the operands' rows must not be read into the product
    check_product(fgb().mxfp4_gemm(a, sa, b, sb, out_dtype=torch.float32), av, bv)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M", [3, 100, 270])
def test_gemm_strides_accumulate_and_edges_of_d(fmt, M):
    N, K = 203, 384
    a, sa, av = operand_a(M, K, fmt, 3)
    b, sb, bv = operand_b(N, K, 4)
    wide = torch.full((M, a.shape[1] + 48), 0xFF, dtype=torch.uint8, device=DEV)
    wide[:, 16:16 + a.shape[1]] = a
    bw = torch.full((N, b.shape[1] + 32), 0xFF, dtype=torch.uint8, device=DEV)
    bw[:, :b.shape[1]] = b
    d = torch.full((M + 2, N + 5), 7.0, device=DEV)
    base = torch.arange(M * N, device=DEV).reshape(M, N).float() / N
    d[1:M + 1, 2:N + 2] = base
    fgb().mxfp4_gemm(wide[:, 16:16 + a.shape[1]], sa, bw[:, :b.shape[1]], sb, a_fmt=FMT[fmt], d=d[1:M + 1, 2:N + 2],
                     accumulate=True)
    check_product(d[1:M + 1, 2:N + 2], av, bv, base.double().cpu().numpy())
    rim = torch.ones_like(d, dtype=torch.bool)
    rim[1:M + 1, 2:N + 2] = False
    assert bool((d[rim] == 7.0).all())
    h = torch.full((M + 2, N + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=FMT[fmt], d=h[1:M + 1, 3:N + 3])
    check_product(h[1:M + 1, 3:N + 3], av, bv)
    rim = torch.ones_like(h, dtype=torch.bool)
    rim[1:M + 1, 3:N + 3] = False
    assert bool((h[rim] == 7.0).all())


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_gemm_empty(fmt):
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    f = FMT[fmt]
    half = 2 if fmt == "e2m1" else 1
    sa = (lambda M, K: u8((K + 255) // 256, M, 8)) if fmt == "e2m1" else (lambda M, K: u8(M, K // 128))
    assert fgb().mxfp4_gemm(u8(0, 256 // half), sa(0, 256), u8(5, 128), u8(1, 5, 8), a_fmt=f).shape == (0, 5)
    assert fgb().mxfp4_gemm(u8(4, 256 // half), sa(4, 256), u8(0, 128), u8(1, 0, 8), a_fmt=f).shape == (4, 0)
    for M in (4, 400):
        d = fgb().mxfp4_gemm(u8(M, 0), sa(M, 0), u8(5, 0), u8(0, 5, 8), a_fmt=f, out_dtype=torch.float32)
        assert bool((d == 0).all()) and d.shape == (M, 5)
        d = torch.ones((M, 5), device=DEV)
        fgb().mxfp4_gemm(u8(M, 0), sa(M, 0), u8(5, 0), u8(0, 5, 8), a_fmt=f, d=d, accumulate=True)
        assert bool((d == 1).all())


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M", [2, 280])
def test_gemm_nan_scale_stays_in_its_row_and_column(fmt, M):
    N, K = 96, 512
    a, sa, av = operand_a(M, K, fmt, 5)
    b, sb, bv = operand_b(N, K, 6)
    sb[1, 40, 3] = 255
    d = fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=FMT[fmt], out_dtype=torch.float32)
    assert bool(torch.isnan(d[:, 40]).all())
    keep = [n for n in range(N) if n != 40]
    check_product(d[:, keep], av, bv[keep])


def test_gemm_far_apart_scales():
    """Groups 2^40 apart: the small ones' products vanish against the large, exactly as in FP32."""
    M, N, K = 40, 64, 1024
    g = torch.Generator().manual_seed(9)
    x = torch.randn((M, K), generator=g) * torch.exp2(torch.randint(-20, 21, (M, K // 32), generator=g)
                                                      .float()).repeat_interleave(32, 1)
    q, s = O.quant(x.double().numpy())
    b, sb, bv = operand_b(N, K, 8)
    d = fgb().mxfp4_gemm(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), b, sb, out_dtype=torch.float32)
    check_product(d, O.dequant(q, s), bv)


def test_linear_training_step():
    """y, dx and dw of a Linear from both directions' copies, tokens that no group divides."""
    T, I, J = 333, 416, 288
    x, w, dy = values(T, I, 1, torch.bfloat16), values(J, I, 2, torch.bfloat16, 2), values(T, J, 3, torch.bfloat16)
    m = fgb()
    xq, xs, xqt, xst = m.mxfp4_quant_t(x.to(DEV))
    wq, ws, wqt, wst = m.mxfp4_quant_t(w.to(DEV))
    gq, gs, gqt, gst = m.mxfp4_quant_t(dy.to(DEV))
    val = lambda t: O.dequant(*O.quant(t.double().numpy()))  # noqa: E731
    check_product(m.mxfp4_gemm(xq, xs, wq, ws), val(x), val(w))
    check_product(m.mxfp4_gemm(gq, gs, wqt, wst), val(dy), val(w.t()))
    check_product(m.mxfp4_gemm(gqt, gst, xqt, xst, out_dtype=torch.float32), val(dy.t()), val(x.t()))


# ---- experts' products ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("rows,N,K", [
    ([1], 64, 128), ([0, 0, 3, 0], 96, 256), ([16, 0, 16, 16], 130, 384), ([5, 40, 0, 1, 200], 200, 640),
    ([300, 0, 257, 7], 260, 256), ([0, 0], 64, 128), ([600, 1, 700], 520, 512),
    ([3] * 70 + [0] * 60, 48, 128),
])
def test_grouped_gemm(rows, N, K, fmt):
    say("grouped", rows[:8], N, K, fmt)
    G, off = len(rows), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    cap = int(off[-1]) + 37
    a, sa, av = operand_a(cap, K, fmt, 11)
    ws = [operand_b(N, K, 20 + g) for g in range(G)]
    b, sb = torch.stack([w[0] for w in ws]), torch.stack([w[1] for w in ws])
    d = torch.full((cap, N), 3.0, dtype=torch.bfloat16, device=DEV)
    out = fgb().mxfp4_grouped_gemm(a, sa, b, sb, torch.from_numpy(off).to(DEV), a_fmt=FMT[fmt], d=d)
    assert out is d and bool((d[off[-1]:] == 3.0).all())
    f = fgb().mxfp4_grouped_gemm(a, sa, b, sb, torch.from_numpy(off).to(DEV), a_fmt=FMT[fmt], out_dtype=torch.float32)
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        if hi > lo:
            check_product(d[lo:hi], av[lo:hi], ws[g][2])
            check_product(f[lo:hi], av[lo:hi], ws[g][2])


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(50, 24600, 384), (64, 24576, 128), (201, 7170, 640)])
def test_gemm_wide_blocks(M, N, K, fmt):
    """Many columns at 33 rows or more: 64 x 128 blocks, with odd rows, columns and K."""
    say("gemm", M, N, K, fmt)
    a, sa, av = operand_a(M, K, fmt, 5)
    b, sb, bv = operand_b(N, K, 6)
    check_product(fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=FMT[fmt], out_dtype=torch.float32), av, bv)
    check_product(fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=FMT[fmt]), av, bv)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_grouped_gemm_wide_blocks(fmt):
    """As many experts as make 64 x 128 blocks of few columns, of 0 to 130 rows."""
    test_grouped_gemm([0, 48, 64, 65, 130, 16, 1, 63] * 8, 400, 384, fmt)


def test_other_streams():
    """Calls on a side stream, ordered after the tensors' own: the same bits."""
    x, w = values(200, 512, 1, torch.bfloat16).to(DEV), values(300, 512, 2, torch.bfloat16).to(DEV)
    m = fgb()
    want = m.mxfp4_gemm(*m.mxfp4_quant(x), *m.mxfp4_quant(w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = m.mxfp4_gemm(*m.mxfp4_quant(x), *m.mxfp4_quant(w))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want, got)
