"""RMSNorm into FP8, the router with a bias and groups, and gradient clipping without a GPU: the 64-bit references
pinned to hand-worked values and to differences, and what the entry points refuse, on the host, before anything is
enqueued."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import norm as N
from oracle import router as R


# ---- the references ------------------------------------------------------------------

def test_norm_by_hand():
    y, rstd = N.forward([[3.0, 4.0], [0.0, 0.0]], [1.0, 2.0], 12.5)
    assert rstd.tolist() == [0.2, 12.5 ** -0.5] and np.allclose(y, [[0.6, 1.6], [0, 0]], rtol=1e-15)


def test_norm_gradient_is_the_difference():
    rng = np.random.default_rng(0)
    h, w, dy, dh = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    eps, step = 0.01, 1e-6

    def objective(h, w):
        return float((N.forward(h, w, eps)[0] * dy).sum() + (h * dh).sum())
    dx, dw = N.backward(dy, h, w, N.forward(h, w, eps)[1], dh)
    for r in range(3):
        for c in range(8):
            up, dn = h.copy(), h.copy()
            up[r, c] += step
            dn[r, c] -= step
            assert abs((objective(up, w) - objective(dn, w)) / (2 * step) - dx[r, c]) < 1e-7
    for c in range(8):
        up, dn = w.copy(), w.copy()
        up[c] += step
        dn[c] -= step
        assert abs((objective(h, up) - objective(h, dn)) / (2 * step) - dw[c]) < 1e-7


def test_choice_by_hand():
    # scores 1/2 each: the bias decides; groups {0,1} {2,3} {4,5} have the values .6+.5, .9+.1, .8+.7
    z = np.zeros((1, 6))
    b = np.array([0.1, 0.0, 0.4, -0.4, 0.3, 0.2], np.float32)
    assert R.choose(z, 3, R.SIGMOID, b).tolist() == [[2, 4, 5]]
    assert R.choose(z, 3, R.SIGMOID, b, 3, 2).tolist() == [[4, 5, 0]]
    assert R.choose(z, 2, R.SIGMOID, b, 3, 1).tolist() == [[4, 5]]
    # without a bias a group's value is its largest logit: {2,3} wins by 0.9
    z = np.array([[0.6, 0.5, 0.9, 0.1, 0.8, 0.7]])
    assert R.choose(z, 3, R.SOFTMAX, None, 3, 2).tolist() == [[2, 4, 5]]
    assert R.choose(z, 2, R.SOFTMAX, None, 3, 1).tolist() == [[2, 3]]
    # equal everywhere: the lowest groups and experts; a group with nothing usable is never chosen
    assert R.choose(np.zeros((1, 6)), 4, R.SOFTMAX, None, 3, 2).tolist() == [[0, 1, 2, 3]]
    z = np.array([[-np.inf, np.nan, 0.0, -np.inf, -1.0, -2.0]])
    assert R.choose(z, 3, R.SIGMOID, np.zeros(6), 3, 3).tolist() == [[2, 4, 5]]
    assert R.choose(z, 2, R.SIGMOID, np.zeros(6), 3, 1).tolist() == [[2, -1]]  # 1/2 against .27 + .12
    assert R.choose(z, 1, R.SIGMOID, np.array([0, 0, -np.inf, 0, 0, 0]), mask=[0]).tolist() == [[-1]]


# ---- refusals of the C entry points -----------------------------------------------------

def _fake(a=0x1000):
    return C.c_void_p(a)


def _lib():
    import fine_grained_blockwise_amd as fgb
    return fgb.lib()


def test_norm_refuses():
    L, f = _lib(), _fake()
    base = dict(x=f, xd=1, rows=4, cols=256, ldx=256, r=f, rd=0, ldr=256, w=f, wd=1, eps=1e-6, group=128, h=f, ldh=256,
                rstd=f, q=f, s=f, y=f, yd=1, ldy=256)

    def n(**kw):
        v = dict(base, **kw)
        return L.rmsnorm_quant(v["x"], v["xd"], v["rows"], v["cols"], v["ldx"], v["r"], v["rd"], v["ldr"], v["w"],
                               v["wd"], v["eps"], v["group"], v["h"], v["ldh"], v["rstd"], v["q"], v["s"], v["y"],
                               v["yd"], v["ldy"], None)
    assert n(x=None) == 1 and b"null" in L.fgb_last_error()
    assert n(xd=2) == 2 and n(rd=2) == 2 and n(wd=2) == 2 and n(yd=2) == 2 and n(group=64) == 2
    assert n(cols=200) == 1 and n(cols=0) == 1 and n(cols=32800, ldx=32800, ldr=32800) == 1 and n(rows=-1) == 1
    assert n(cols=160, ldx=160, ldr=160, ldh=160, ldy=160) == 1  # no multiple of the group
    assert n(ldx=248) == 1 and n(ldx=257) == 1 and n(ldr=250) == 1 and n(ldh=128) == 1 and n(ldy=260) == 1
    assert n(x=_fake(0x1008)) == 1 and n(w=_fake(0x1002)) == 1 and n(h=_fake(0x1004)) == 1 and n(q=_fake(0x1008)) == 1
    assert n(h=None) == 1 and n(rstd=None) == 1 and n(rstd=_fake(0x1002)) == 1 and n(w=None) == 1
    assert n(q=None) == 1 and n(s=None) == 1 and n(q=None, s=None, y=None) == 1
    assert n(eps=0.0) == 1 and n(eps=-1.0) == 1 and n(eps=float("nan")) == 1 and n(eps=1e-60) == 1
    assert n(rows=0, x=None, h=None, rstd=None) == 0


def test_norm_backward_refuses():
    L, f = _lib(), _fake()
    need = L.rmsnorm_backward_workspace_size(4, 256)
    assert need >= 4 * 256 and L.rmsnorm_backward_workspace_size(-1, 256) == 0
    assert L.rmsnorm_backward_workspace_size(4, 32800) == 0
    base = dict(dy=f, dd=1, rows=4, cols=256, lddy=256, h=f, hd=1, ldh=256, w=f, wd=0, rstd=f, dh=f, lddh=256, dx=f,
                lddx=256, dw=f, ws=f, n=need)

    def b(**kw):
        v = dict(base, **kw)
        return L.rmsnorm_backward(v["dy"], v["dd"], v["rows"], v["cols"], v["lddy"], v["h"], v["hd"], v["ldh"], v["w"],
                                  v["wd"], v["rstd"], v["dh"], v["lddh"], v["dx"], v["lddx"], v["dw"], v["ws"], v["n"],
                                  None)
    for k in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert b(**{k: None}) == 1, k
        assert b(**{k: _fake(0x1002)}) == 1, k
    assert b(dd=2) == 2 and b(hd=3) == 2 and b(wd=2) == 2 and b(cols=250) == 1 and b(rows=-1) == 1
    assert b(lddy=255) == 1 and b(ldh=128) == 1 and b(lddh=260) == 1 and b(lddx=4) == 1 and b(dh=_fake(0x1004)) == 1
    assert b(ws=None) == 3 and b(n=need - 1) == 3 and b(ws=_fake(0x1008)) == 1


def test_grouped_router_refuses():
    L, f = _lib(), _fake()
    ws = L.moe_router_workspace_size(64, 24)
    base = dict(z=f, dt=0, T=64, E=24, ld=24, k=4, bias=f, G=4, kg=2, score=1, idx=f, w=f, counts=f, ws=f, n=ws)

    def r(**kw):
        v = dict(base, **kw)
        return L.moe_router_grouped(v["z"], v["dt"], v["T"], v["E"], v["ld"], v["k"], None, v["bias"], v["G"], v["kg"],
                                    v["score"], 1, 1.0, 0.0, v["idx"], v["w"], v["counts"], None, v["ws"], v["n"], None)
    assert r(G=5) == 1 and r(G=0) == 1 and r(G=-4) == 1 and r(kg=0) == 1 and r(kg=5) == 1 and r(k=13) == 1
    assert b"topk_groups" in L.fgb_last_error()
    assert r(E=128, ld=128, G=128, kg=8) == 1 and r(bias=_fake(0x1002)) == 1
    assert r(z=None) == 1 and r(dt=2) == 2 and r(score=2) == 2 and r(ld=23) == 1 and r(idx=None) == 1
    assert r(ws=None) == 3 and r(n=ws - 1) == 3
    assert L.moe_bias_update(f, f, 0, 1e-3, f, None) == 1 and L.moe_bias_update(f, f, 1025, 1e-3, f, None) == 1
    assert L.moe_bias_update(None, f, 8, 1e-3, f, None) == 1 and L.moe_bias_update(f, f, 8, 1e-3, _fake(0x1002), None) == 1


def _arr(kind, *v):
    return (kind * len(v))(*v)


def test_clip_refuses():
    L, f = _lib(), _fake()
    P, I = C.c_void_p, C.c_int64

    def c(g=(0x1000, 0x9000), o=(0x1000, 0x9000), n=(8, 8), t=(0, 0), u=(0, 0), most=1.0, scale=1.0, sumsq=f, norm=f,
          ws=f, wn=1 << 20, count=None):
        return L.grad_clip(_arr(P, *g), _arr(P, *o), _arr(I, *n), _arr(C.c_int, *t), _arr(C.c_int, *u),
                           len(g) if count is None else count, most, scale, sumsq, norm, ws, wn, None)
    assert c(t=(0, 2)) == 2 and c(u=(3, 0)) == 2 and c(n=(8, -1)) == 1 and c(n=(8, 1 << 41)) == 1
    assert c(g=(0, 0x9000)) == 1 and c(o=(0x1000, 0)) == 1 and c(g=(0x1002, 0x9000)) == 1 and c(o=(0x1000, 0x9002)) == 1
    for bad in (0.0, -1.0, float("nan")):
        assert c(most=bad) == 1 and c(scale=bad) == 1
    assert c(scale=float("inf")) == 1 and c(norm=None) == 1 and c(norm=_fake(0x1002)) == 1 and c(sumsq=_fake(0x1004)) == 1
    assert c(sumsq=None, ws=None) == 3 and c(sumsq=None, wn=8) == 3 and c(sumsq=None, ws=_fake(0x1004)) == 1
    assert c(count=-1) == 1
    # an output over another output, over another's gradient, half over its own, over its own in another type
    assert c(o=(0x2000, 0x2000)) == 1 and b"lies over" in L.fgb_last_error()
    assert c(o=(0x2000, 0x201C)) == 1 and c(o=(0x9000, 0x2000)) == 1 and c(o=(0x1010, 0x9000)) == 1
    assert c(u=(1, 0)) == 1 and c(g=(0x1000, 0x1000), o=(0x1000, 0x2000)) == 1
    assert c(g=(0x1000, 0x1010), o=(0x1000, 0x2000)) == 1 and c(o=(0x2000, 0x8FF0)) == 1
    # a long output that starts before a short one inside it
    assert c(g=(0x1000, 0x9000, 0x9100), o=(0x2000, 0x2100, 0x2300), n=(256, 4, 4), t=(0,) * 3, u=(0,) * 3) == 1

    def s(g=(0x1000,), n=(8,), t=(0,), out=f, ws=f, wn=16):
        return L.grad_sumsq(_arr(P, *g), _arr(I, *n), _arr(C.c_int, *t), 1, out, 0, ws, wn, None)
    assert s(out=None) == 1 and s(out=_fake(0x1004)) == 1 and s(ws=None) == 3 and s(wn=8) == 3 and s(t=(7,)) == 2
    assert s(g=(0x1001,), t=(1,)) == 1 and L.grad_sumsq(None, None, None, 3, f, 0, f, 64, None) == 1


def test_clip_workspace_counts_launches():
    import fine_grained_blockwise_amd as fgb
    size = fgb.grad_sumsq_workspace_size
    assert size([0, 0]) == 8 and size([1]) == 16 and size([1, 0, 1]) == 24
    assert size([1] * 1000) == 8 * 1001 and size([1 << 34]) == size([1 << 35])


# ---- refusals of the binding -----------------------------------------------------------------

def test_binding_refuses():
    import fine_grained_blockwise_amd as fgb
    x, w = torch.zeros(4, 256), torch.zeros(256)
    for kw, what in ((dict(group=64), "group"), (dict(quant=False), "y_dtype"), (dict(eps=0.0), "eps"),
                     (dict(h=x), "residual")):
        with pytest.raises(ValueError, match=what):
            fgb.rmsnorm_quant(x, w, **kw)
    with pytest.raises(ValueError, match="GPU"):
        fgb.rmsnorm_quant(x, w)
    with pytest.raises(ValueError, match="2-D"):
        fgb.rmsnorm_quant(w, w)
    with pytest.raises(TypeError):
        fgb.rmsnorm_quant(x.half(), w)
    with pytest.raises(ValueError, match="GPU"):
        fgb.rmsnorm_backward(x, x, w, torch.zeros(4))
    z = torch.zeros(4, 24)
    for kw, what in ((dict(groups=5), "groups"), (dict(groups=0), "groups"), (dict(groups=4, topk_groups=5), "topk_groups"),
                     (dict(groups=12, topk_groups=1), "topk_groups"), (dict(bias=torch.zeros(23)), "bias"),
                     (dict(bias=torch.zeros(24, dtype=torch.float64)), "bias"), (dict(bias=torch.zeros(24)), "GPU")):
        with pytest.raises(ValueError, match=what):
            fgb.moe_router(z, 4, **kw)
    with pytest.raises(ValueError, match="counts"):
        fgb.moe_bias_update(torch.zeros(8), torch.zeros(8, dtype=torch.int32), 1e-3)
    with pytest.raises(ValueError, match="GPU"):
        fgb.moe_bias_update(torch.zeros(8), torch.zeros(9, dtype=torch.int32), 1e-3)
    for call in (lambda g: fgb.grad_clip(g, 1.0), fgb.grad_sumsq):
        with pytest.raises(ValueError, match="GPU"):
            call([torch.zeros(4)])
        with pytest.raises(ValueError, match="empty"):
            call([])


def test_calls_run_on_their_tensors_device(monkeypatch):
    """A launch goes to the current device, so a call for another one makes that current."""
    import fine_grained_blockwise_amd as fgb
    seen = []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            seen.append(("enter", self.d.index))

        def __exit__(self, *a):
            seen.append(("exit", self.d.index))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(fgb, "_current_device", lambda: 1)
    monkeypatch.setattr(fgb, "_call", lambda *a: seen.append(a))
    fgb._call_on(torch.device("cuda", 1), "f", 2)
    assert seen == [("f", 2)]
    fgb._call_on(torch.device("cuda", 0), "g", 3)
    assert seen[1:] == [("enter", 0), ("g", 3), ("exit", 0)]


def test_tensor_helper():
    import fine_grained_blockwise_amd as fgb
    t = fgb._tensors
    a = t.empties(torch.zeros(2), (0, 3, 4), (1, 5), (2,), (3, 0, 2, 3))
    assert [(v.dtype, tuple(v.shape)) for v in a] == [(torch.float32, (3, 4)), (torch.bfloat16, (5,)),
                                                      (torch.uint8, ()), (torch.int32, (0, 2, 3))]
    for bad in ((torch.zeros(1), 3), (3,), (), (torch.zeros(1), ()), (torch.zeros(1), (0, 1, 1, 1, 1)), (torch.zeros(1), ("x",))):
        with pytest.raises(TypeError):
            t.empties(*bad)
    for bad in ((4, 1), (0, -1)):
        with pytest.raises(ValueError):
            t.empties(torch.zeros(1), bad)
    with pytest.raises(RuntimeError):
        t.empties(torch.zeros(1), (0, 1 << 62, 1 << 62))
    assert t.usual(torch.zeros(2, 3), torch.zeros(3), None) is None and t.usual(None, torch.zeros(3)) is None  # (no GPU)
    with pytest.raises(TypeError):
        t.usual(torch.zeros(2, 3))
    assert t.describe([]) == (b"", b"", b"", -1)
    for bad in (3, [torch.zeros(1), None], [object()]):
        with pytest.raises((TypeError, ValueError)):
            t.describe(bad)
