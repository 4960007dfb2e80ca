"""MXFP4 and router without a GPU: the 64-bit references pinned to hand-worked values and to differences, and
what the entry points refuse, on the host, before anything is enqueued."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import mxfp4 as O
from oracle import router as R


# ---- the references ------------------------------------------------------------------

def test_e2m1_codes_by_hand():
    v = np.array([0.0, 0.25, 0.26, 0.74, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, 9.0, -0.0, -0.3, -6.0])
    want = [0, 0, 1, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 7, 8, 9, 15]
    assert O.encode(v).tolist() == want


@pytest.mark.parametrize("amax,ceil,floor", [
    (6.0, 0, 0), (6.1, 1, 0), (4.0, 0, 0), (3.99, 0, -1), (3.0, -1, -1), (3.01, 0, -1), (1.0, -2, -2), (0.0, -127, -127),
    (2.0 ** -130, -127, -127), (float(np.float32(3.4e38)), 126, 125),
])
def test_scale_exponents_by_hand(amax, ceil, floor):
    assert O.scale_exp(amax, O.CEIL) == ceil
    assert O.scale_exp(amax, O.FLOOR) == floor


def test_quant_layout_by_hand():
    x = np.zeros((2, 288))
    x[1, 0], x[1, 1], x[0, 33], x[1, 287] = 6.0, -3.0, 12.0, np.inf
    q, s = O.quant(x)
    assert q.shape == (2, 144) and s.shape == (2, 2, 8)
    assert q[1, 0] == (7 | (13 << 4)) and s[0, 1, 0] == 127
    assert q[0, 16] == (7 << 4) and s[0, 0, 1] == 128
    assert s[1, 1, 0] == 255 and s[1, :, 1:].max() == 0 and s[1, 0, 0] == 0
    d = O.dequant(q, s)
    assert d[1, 0] == 6 and d[1, 1] == -3 and d[0, 33] == 12 and np.isnan(d[1, 256:]).all()


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_is_the_objective_s_difference(score, renorm):
    rng = np.random.default_rng(5)
    T, E, k = 5, 7, 3
    z = rng.normal(size=(T, E)) * 1.5
    z[1, 2:] = -np.inf  # fewer experts than slots
    z[3] = -np.inf
    f = R.forward(z, k, score, renorm, 1.7, 0.3, mask=[1, 1, 0, 1, 1])
    assert (f["idx"][2] == -1).all() and (f["idx"][3] == -1).all() and f["idx"][1, 2] == -1 and f["counts"][E] == 3
    dw = rng.normal(size=(T, k))
    how = (f["idx"], f["counts"], dw, 0.8, score, renorm, 1.7, 0.3)
    dz = R.backward(z, *how)
    for t in range(T):
        for e in range(E):
            if np.isfinite(z[t, e]):
                h = 1e-6
                up, dn = z.copy(), z.copy()
                up[t, e] += h
                dn[t, e] -= h
                want = (R.objective(up, *how) - R.objective(dn, *how)) / (2 * h)
                assert abs(want - dz[t, e]) < 1e-8
            else:
                assert dz[t, e] == 0


def test_router_loss_by_hand():
    # two tokens, two experts, top-1, equal logits: both choose expert 0, p = 1/2 each
    f = R.forward(np.zeros((2, 2)), 1, coef=1.0)
    assert f["idx"].ravel().tolist() == [0, 0] and f["counts"].tolist() == [2, 0, 2]
    assert f["loss"] == 2 / (1 * 4) * (2 * 1.0)


# ---- refusals ----------------------------------------------------------------------------

def _fake(a=0x1000):
    return C.c_void_p(a)


def test_quant_refuses():
    import fine_grained_blockwise_amd as fgb
    L, f = fgb.lib(), _fake()

    def q(x=f, dt=1, G=1, rows=4, cols=64, ld=64, rule=0, q=f, s=f):
        return L.mxfp4_quant(x, dt, G, rows, cols, ld, rule, q, s, None)

    def qt(x=f, dt=1, G=1, rows=4, cols=64, ld=64, rule=0, qt=f, st=f):
        return L.mxfp4_quant_t(x, dt, G, rows, cols, ld, rule, f, f, qt, st, None)
    for call in (q, qt):
        assert call(x=None) == 1 and b"null" in L.fgb_last_error()
        assert call(dt=3) == 2 and call(rule=2) == 2
        assert call(cols=48) == 1 and call(rows=-1) == 1 and call(ld=32) == 1 and call(ld=68) == 1
        assert call(x=_fake(0x1008)) == 1 and b"aligned" in L.fgb_last_error()
        assert call(rows=0, x=None) == 0 and call(cols=0, x=None) == 0 and call(G=0) == 0
        assert call(rows=1 << 31) == 1
    assert q(s=None) == 1 and q(q=_fake(0x1004)) == 1
    assert qt(st=None) == 1 and qt(qt=_fake(0x1004)) == 1 and qt(rows=1 << 24) == 1

    def dq(q=f, s=f, rows=4, cols=64, out=f, dt=1):
        return L.mxfp4_dequant(q, s, rows, cols, out, dt, None)
    assert dq(q=None) == 1 and dq(cols=40) == 1 and dq(dt=2) == 2 and dq(out=_fake(0x1004)) == 1 and dq(rows=0) == 0


def test_gemm_refuses():
    import fine_grained_blockwise_amd as fgb
    L, f = fgb.lib(), _fake()
    base = dict(a=f, sa=f, fmt=2, b=f, sb=f, M=64, N=64, K=128, lda=64, ldb=64, d=f, dt=1, ldd=64, acc=0)

    def g(**kw):
        v = dict(base, **kw)
        return L.mxfp4_gemm(v["a"], v["sa"], v["fmt"], v["b"], v["sb"], v["M"], v["N"], v["K"], v["lda"], v["ldb"],
                            v["d"], v["dt"], v["ldd"], v["acc"], None)
    assert g(fmt=1) == 2 and g(fmt=7) == 2 and g(dt=2) == 2
    assert g(K=48) == 1 and g(fmt=0, K=96, lda=96) == 1 and g(M=-1) == 1
    assert g(lda=48) == 1 and g(ldb=72) == 1 and g(ldd=63) == 1 and g(lda=1 << 25) == 1
    assert g(a=None) == 1 and g(sb=None) == 1 and g(d=None) == 1
    assert g(a=_fake(0x1008)) == 1 and g(sa=_fake(0x1008)) == 1 and g(d=_fake(0x1001)) == 1
    assert g(acc=1) == 2
    assert g(dt=0, ldd=1 << 23) == 2
    assert g(M=0, a=None, d=None) == 0 and g(N=0, d=None) == 0

    def gg(a=f, fmt=0, off=f, G=4, M=64, N=64, K=128, d=f, dt=1):
        return L.mxfp4_grouped_gemm(a, f, fmt, f, f, off, G, M, N, K, d, dt, None)
    assert gg(off=None) == 1 and gg(G=0) == 1 and gg(G=1025) == 1 and gg(K=64) == 1 and gg(fmt=3) == 2
    assert gg(d=None) == 1 and gg(dt=5) == 2 and gg(M=0) == 0 and gg(a=_fake(0x1004)) == 1
    assert gg(dt=0, N=1 << 23) == 2


def test_router_refuses():
    import fine_grained_blockwise_amd as fgb
    L, f = fgb.lib(), _fake()
    ws = fgb.moe_router_workspace_size(64, 8)
    assert ws > 0 and fgb.moe_router_workspace_size(-1, 8) == 0 and fgb.moe_router_workspace_size(4, 2000) == 0
    base = dict(z=f, dt=0, T=64, E=8, ld=8, k=2, score=0, idx=f, w=f, counts=f, ws=f, n=ws)

    def r(**kw):
        v = dict(base, **kw)
        return L.moe_router(v["z"], v["dt"], v["T"], v["E"], v["ld"], v["k"], None, v["score"], 0, 1.0, 0.0, v["idx"],
                            v["w"], v["counts"], None, v["ws"], v["n"], None)
    assert r(z=None) == 1 and r(dt=2) == 2 and r(score=2) == 2
    assert r(E=0) == 1 and r(E=1025, ld=1025) == 1 and r(k=0) == 1 and r(k=9) == 1 and r(E=100, ld=100, k=65) == 1
    assert r(ld=7) == 1 and r(T=-1) == 1 and r(z=_fake(0x1002)) == 1
    assert r(idx=None) == 1 and r(counts=None) == 1 and r(w=_fake(0x1002)) == 1
    assert r(ws=None) == 3 and r(n=ws - 1) == 3 and b"workspace" in L.fgb_last_error()

    def b(z=f, dt=1, idx=f, counts=f, dz=f, ldd=8, k=2):
        return L.moe_router_backward(z, dt, 64, 8, 8, k, idx, counts, None, None, 0, 0, 1.0, 0.0, dz, ldd, None)
    assert b(idx=None) == 1 and b(counts=None) == 1 and b(dz=None) == 1 and b(ldd=7) == 1 and b(k=9) == 1 and b(dt=4) == 2
    assert b(dz=_fake(0x1001)) == 1
    assert L.moe_router_backward(None, 0, 0, 8, 8, 2, None, None, None, None, 0, 0, 1.0, 0.0, None, 8, None) == 0


def test_binding_refuses():
    import fine_grained_blockwise_amd as fgb
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError, match="multiple of 32"):
        fgb.mxfp4_quant(torch.zeros(2, 40))
    with pytest.raises(TypeError):
        fgb.mxfp4_quant(torch.zeros(2, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        fgb.mxfp4_quant(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="shape"):
        fgb.mxfp4_dequant(u8(2, 32), u8(1, 2, 2))
    with pytest.raises(ValueError, match="same K"):
        fgb.mxfp4_gemm(u8(2, 32), u8(1, 2, 8), u8(3, 16), u8(1, 3, 8))
    with pytest.raises(ValueError, match="a_fmt"):
        fgb.mxfp4_gemm(u8(2, 32), u8(1, 2, 8), u8(3, 32), u8(1, 3, 8), a_fmt=fgb.E5M2)
    with pytest.raises(ValueError, match="group_offsets"):
        fgb.mxfp4_grouped_gemm(u8(2, 128), u8(2, 1), u8(3, 5, 64), u8(3, 1, 5, 8), torch.zeros(3, dtype=torch.int32))
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="topk"):
        fgb.moe_router(z, 9)
    with pytest.raises(ValueError, match="stride"):
        fgb.moe_router(torch.zeros(8, 4).t(), 2)
    with pytest.raises(ValueError, match="token_mask"):
        fgb.moe_router(z, 2, token_mask=torch.zeros(4))
    with pytest.raises(ValueError, match="counts"):
        fgb.moe_router_backward(z, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32))
