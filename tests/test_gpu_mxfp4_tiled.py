"""The MXFP4 products on the 256 x 256-tiled kernel, at sizes that the library says it takes there (asserted, so that
another rule of choice cannot empty these tests): several steps of K with tails, ragged tiles, FP32 sums onto D, strided
operands and outputs, NaN scales, experts with unpadded segments.  The whole of D is compared with the product of the
operands' values in 64 bits, within the bound of K products summed in FP32, K 2^-24 sum |product|, one rounding of
the result, and half a BF16 ulp more where D is BF16."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def fgb():
    import fine_grained_blockwise_amd as m
    return m


def say(*a):
    print("[case]", *a, flush=True)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def e2m1(rows, K, seed):
    """Random codes and scales 2^-6 .. 2^6 of a [rows, K] MXFP4 tensor, and its values."""
    g = gen(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    e = torch.randint(-6, 7, (rows, K // 32), generator=g, device=DEV)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -(K // 32) % 8))
    s = s.view(rows, -1, 8).transpose(0, 1).contiguous()
    code = torch.stack((q & 15, q >> 4), 2).view(rows, K).long()
    v = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64, device=DEV)[code]
    return q, s, (v.view(rows, -1, 32) * torch.exp2(e.double())[..., None]).view(rows, K)


def e4m3(rows, K, seed):
    """Random E4M3 codes (no NaN) with scales 2^-6 .. 2^6 per 128 columns, and their values."""
    g = gen(seed)
    q = torch.randint(0, 127, (rows, K), generator=g, dtype=torch.uint8, device=DEV)
    q |= torch.randint(0, 2, (rows, K), generator=g, dtype=torch.uint8, device=DEV) << 7
    e = torch.randint(-6, 7, (rows, K // 128), generator=g, device=DEV)
    v = q.view(torch.float8_e4m3fn).double().view(rows, -1, 128) * torch.exp2(e.double())[..., None]
    return q, (e + 127).to(torch.uint8), v.view(rows, K)


def operand_a(fmt, rows, K, seed):
    return (e2m1 if fmt == "e2m1" else e4m3)(rows, K, seed)


def code(fmt):
    return fgb().E2M1 if fmt == "e2m1" else fgb().E4M3


def check(got, av, bv, base=0.0):
    ref, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    tol = av.shape[1] * 2.0 ** -24 * mag + 2.0 ** -24 * (ref.abs() + torch.as_tensor(base).abs()) + 1e-44
    ref = ref + base
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -134
    ratio = ((got.double() - ref).abs() / tol).max()
    assert float(ratio) <= 1.0, float(ratio)  # (a NaN fails)


def tiled(M, N, K, fmt, groups=0):
    say("tiled", M, N, K, fmt, groups)
    assert fgb().mxfp4_gemm_tiled(M, N, K, a_fmt=code(fmt), groups=groups)


# two operands in MXFP4: steps of 256, K in units of 32; an E4M3 A: steps of 128
DENSE = [("e2m1", 4095, 4093, 224), ("e2m1", 4093, 4095, 256), ("e2m1", 4097, 3811, 288), ("e2m1", 3301, 3585, 512),
         ("e2m1", 2049, 2309, 1056), ("e2m1", 2303, 2049, 1248), ("e2m1", 1537, 2830, 2304), ("e2m1", 2305, 1281, 4064),
         ("e4m3", 3841, 3585, 256), ("e4m3", 3301, 3585, 384), ("e4m3", 2049, 2309, 1152),
         ("e4m3", 2305, 2817, 1280), ("e4m3", 2049, 2561, 3968)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt,M,N,K", DENSE)
def test_gemm(fmt, M, N, K, out):
    tiled(M, N, K, fmt)
    a, sa, av = operand_a(fmt, M, K, 1)
    b, sb, bv = e2m1(N, K, 2)
    d = fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=code(fmt), out_dtype=out)
    check(d, av, bv)
    assert torch.equal(d, fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=code(fmt), out_dtype=out))


@pytest.mark.parametrize("fmt,M,N,K", [("e2m1", 2049, 2309, 1120), ("e4m3", 2305, 2817, 1280)])
def test_strides_accumulate_and_edges_of_d(fmt, M, N, K):
    tiled(M, N, K, fmt)
    m = fgb()
    a, sa, av = operand_a(fmt, M, K, 3)
    b, sb, bv = e2m1(N, K, 4)
    row = a.shape[1]
    wide = torch.full((M, (row + 15) // 16 * 16 + 48), 0xFF, dtype=torch.uint8, device=DEV)
    wide[:, 16:16 + row] = a
    bw = torch.full((N, K // 2 + 32), 0xFF, dtype=torch.uint8, device=DEV)
    bw[:, :K // 2] = b
    base = torch.arange(M * N, device=DEV).reshape(M, N).float() / N
    for dtype, acc in ((torch.float32, True), (torch.float32, False), (torch.bfloat16, False)):
        d = torch.full((M + 2, N + 5), 7.0, dtype=dtype, device=DEV)
        view = d[1:M + 1, 3:N + 3]
        view.copy_(base)
        m.mxfp4_gemm(wide[:, 16:16 + row], sa, bw[:, :K // 2], sb, a_fmt=code(fmt), d=view, accumulate=acc)
        check(view, av, bv, base.double() if acc else 0.0)
        rim = torch.ones_like(d, dtype=torch.bool)
        rim[1:M + 1, 3:N + 3] = False
        assert bool((d[rim] == 7.0).all())


@pytest.mark.parametrize("fmt,M,N,K", [("e2m1", 2049, 2309, 1120), ("e4m3", 2305, 2817, 1280)])
def test_nan_scales_stay_in_their_row_and_column(fmt, M, N, K):
    tiled(M, N, K, fmt)
    a, sa, av = operand_a(fmt, M, K, 5)
    b, sb, bv = e2m1(N, K, 6)
    sb[2, 300, 5] = 255
    rows = torch.ones(M, dtype=torch.bool, device=DEV)
    if fmt == "e2m1":
        sa[1, 777, 3] = 255
        rows[777] = False
    d = fgb().mxfp4_gemm(a, sa, b, sb, a_fmt=code(fmt), out_dtype=torch.float32)
    assert bool(torch.isnan(d[:, 300]).all()) and bool(torch.isnan(d[~rows]).all())
    cols = torch.ones(N, dtype=torch.bool, device=DEV)
    cols[300] = False
    check(d[rows][:, cols], av[rows], bv[cols])


@pytest.mark.parametrize("fmt,rows,N,K", [
    ("e2m1", [0, 1301, 257, 0, 1, 2500, 301], 2309, 1056), ("e2m1", [700, 13, 0, 900, 1555, 256], 2305, 2272),
    ("e2m1", [130] * 66, 2049, 2048), ("e4m3", [0, 1301, 257, 0, 1, 2500, 301], 2309, 1152),
    ("e4m3", [700, 13, 0, 900, 1555, 256], 2305, 1280), ("e4m3", [301] * 66, 2049, 2048),
])
def test_grouped(fmt, rows, N, K):
    m, G, cap = fgb(), len(rows), sum(rows) + 133
    tiled(cap, N, K, fmt, G)
    off = [0]
    for r in rows:
        off.append(off[-1] + r)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    a, sa, av = operand_a(fmt, cap, K, 7)
    b, sb, bv = e2m1(G * N, K, 8)
    b, bv = b.view(G, N, -1), bv.view(G, N, K)
    sb = sb.view(-1, G, N, 8).transpose(0, 1).contiguous()
    d = torch.full((cap, N), 3.0, dtype=torch.bfloat16, device=DEV)
    m.mxfp4_grouped_gemm(a, sa, b, sb, offs, a_fmt=code(fmt), d=d)
    f = torch.full((cap, N), 3.0, device=DEV)
    m.mxfp4_grouped_gemm(a, sa, b, sb, offs, a_fmt=code(fmt), d=f)
    assert bool((d[off[-1]:] == 3.0).all()) and bool((f[off[-1]:] == 3.0).all())
    for g in range(G):
        if off[g + 1] > off[g]:
            part = slice(off[g], off[g + 1])
            check(d[part], av[part], bv[g])
            check(f[part], av[part], bv[g])


def test_linear_training_step():
    """y, dx and dw from both directions' copies, a number of tokens that no group divides."""
    m = fgb()
    T, I, J = 2085, 2336, 2112
    for M, N, K in ((T, J, I), (T, I, J), (J, I, (T + 31) // 32 * 32)):
        tiled(M, N, K, "e2m1")
    x, w, dy = (torch.randn(s, generator=gen(9 + i), device=DEV).bfloat16()
                for i, s in enumerate(((T, I), (J, I), (T, J))))
    xq, xs, xqt, xst = m.mxfp4_quant_t(x)
    wq, ws, wqt, wst = m.mxfp4_quant_t(w)
    gq, gs, gqt, gst = m.mxfp4_quant_t(dy)
    val = lambda q, s: m.mxfp4_dequant(q, s).double()  # noqa: E731
    check(m.mxfp4_gemm(xq, xs, wq, ws), val(xq, xs), val(wq, ws))
    check(m.mxfp4_gemm(gq, gs, wqt, wst), val(gq, gs), val(wqt, wst))
    dw = m.mxfp4_gemm(gqt, gst, xqt, xst, out_dtype=torch.float32)
    check(dw, val(gqt, gst), val(xqt, xst))


@pytest.mark.parametrize("fmt,M,N,K", [("e2m1", 2049, 2309, 1120), ("e4m3", 2305, 2817, 1280)])
def test_in_a_graph(fmt, M, N, K):
    """Captured once, replayed on other activations with eager work between: the eager result's bits."""
    tiled(M, N, K, fmt)
    m = fgb()
    a, sa, _ = operand_a(fmt, M, K, 1)
    b, sb, _ = e2m1(N, K, 2)
    m.mxfp4_gemm(a, sa, b, sb, a_fmt=code(fmt))  # once eagerly before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = m.mxfp4_gemm(a, sa, b, sb, a_fmt=code(fmt))
    for seed in (1, 3, 4):
        for t, new in zip((a, sa), operand_a(fmt, M, K, seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got, want = held.clone(), m.mxfp4_gemm(a, sa, b, sb, a_fmt=code(fmt))
        assert torch.equal(got, want)
