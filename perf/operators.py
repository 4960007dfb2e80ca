"""Cases of the MoE router and of the MXFP4 quantiser and products, for timing and comparison.

Every case names an operation and its sizes:

  route    the router's forward pass (serving): the experts of each token, their weights, the slots per expert
  train    the router's forward and backward pass: the balance loss and the gradient of the logits too
  quant    MXFP4 quantisation of a tensor (and, with both = True, of its transpose); returns the values
           that the codes and scales stand for
  linear   a product of fresh activations with MXFP4 weights: activations quantised to MXFP4 ("e2m1") or at
           hand as E4M3 codes with 1x128 scales ("e4m3")
  step     a Linear's training step in MXFP4: both directions of x, w and dy quantised, then y, dx and dw
  experts  one product of every token row with the MXFP4 weights of its expert, the rows grouped by expert
           and padded to 16 as permute_pad leaves them, E4M3 codes with 1x128 scales

MXFP4: E2M1 codes, two to a byte (even column in the low half), and one scale byte b = e + 127 for each 32
columns of a row, meaning 2^e.  Scales lie as [ceil(cols / 256), rows, 8]: byte j of entry (i, r) belongs to
columns 256 i + 32 j .. + 31 of row r; bytes past the last column are 0.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decode step through a 32-expert router
        dict(name="route_token", op="route", T=1, E=32, k=8, score="softmax", renorm=True, dtype="f32", masked=False),
        # a training batch of the 32-expert layer
        dict(name="train_16k_e32", op="train", T=16384, E=32, k=8, score="softmax", renorm=True, dtype="f32",
             masked=False),
        # a ragged batch with padding tokens and disabled experts, more experts than a wave has lanes, bf16 logits
        dict(name="train_odd_e257", op="train", T=4999, E=257, k=6, score="sigmoid", renorm=True, dtype="bf16",
             masked=True),
        # one token's hidden state
        dict(name="quant_token", op="quant", rows=1, cols=7168, dtype="bf16", rule="ceil", both=False),
        # an fp32 gradient with a number of tokens that no tile divides, the standard's floor rule, both directions
        dict(name="quant_odd_both", op="quant", rows=1009, cols=2048, dtype="f32", rule="floor", both=True),
        # the activations of a training batch, both directions
        dict(name="quant_8k_both", op="quant", rows=8192, cols=7168, dtype="bf16", rule="ceil", both=True),
        # one token through a projection: decode
        dict(name="linear_token", op="linear", M=1, N=2048, K=7168, act="e2m1", out="bf16"),
        # a short prompt, sizes that no tile divides, E4M3 activations, fp32 out
        dict(name="linear_odd_e4m3", op="linear", M=77, N=2112, K=1536, act="e4m3", out="f32"),
        # a long prompt through a wide projection
        dict(name="linear_4k_wide", op="linear", M=4096, N=28672, K=8192, act="e2m1", out="bf16"),
        # a training step of a dense projection
        dict(name="step_8k", op="step", T=8192, Cin=7168, Cout=2048),
        # one decoded token's eight experts
        dict(name="experts_token", op="experts", T=1, E=32, k=8, N=4096, K=7168),
        # a full batch through all experts' first product
        dict(name="experts_16k", op="experts", T=16384, E=32, k=8, N=4096, K=7168),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        n = step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if n != 3072 else n + step

    op = rng.choice(["route", "train", "quant", "linear", "step", "experts"])
    if op in ("route", "train"):
        E = log(8, 512)
        return dict(op=op, T=log(1, 32768), E=E, k=rng.randint(1, min(8, E)),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5)
    if op == "quant":
        return dict(op=op, rows=log(1, 16384), cols=log(4, 256, 32), dtype=rng.choice(["f32", "bf16"]),
                    rule=rng.choice(["ceil", "floor"]), both=rng.random() < 0.5)
    if op == "linear":
        act = rng.choice(["e2m1", "e4m3"])
        return dict(op=op, M=log(1, 8192), N=log(16, 8192), K=log(4, 224, 32) if act == "e2m1" else log(1, 56, 128),
                    act=act, out=rng.choice(["bf16", "f32"]))
    if op == "step":
        return dict(op=op, T=log(64, 8192), Cin=log(4, 224, 32), Cout=log(4, 224, 32))
    E = log(4, 64)
    return dict(op=op, T=log(1, 8192), E=E, k=rng.randint(1, min(8, E)), N=log(64, 4096), K=log(4, 56, 128))


# ---- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _activations(g, rows, cols, dtype):
    # hidden states: a few channels much larger than the rest
    x = torch.randn((rows, cols), generator=g, device=DEV)
    big = torch.rand((cols,), generator=g, device=DEV) < 0.01
    return torch.where(big, 20.0 * x, x).to(dtype)


def _router_inputs(c, seed):
    g = _gen(seed)
    T, E, k = c["T"], c["E"], c["k"]
    skew = torch.randn((1, E), generator=g, device=DEV)  # some experts are liked more
    z = 1.5 * torch.randn((T, E), generator=g, device=DEV) + skew
    mask = None
    if c["masked"]:
        z[torch.rand((T, E), generator=g, device=DEV) < 0.1] = -math.inf      # experts a token may not use
        z[torch.rand((T,), generator=g, device=DEV) < 0.02] = -math.inf       # tokens with none left
        mask = torch.rand((T,), generator=g, device=DEV) < 0.9                # padding tokens
    st = dict(case=c, logits=z.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16), mask=mask,
              scale=2.5 if c["score"] == "sigmoid" else 1.0, coef=0.01)
    if c["op"] == "train":
        st["dweights"] = _normal(g, (T, k), 1e-2)
        st["dloss"] = torch.ones((), device=DEV)
    return st


def _e4m3_rows(x):
    """E4M3 codes (bytes) and 1x128 power-of-two scale bytes of x [rows, cols]."""
    rows, cols = x.shape
    v = x.float().view(rows, cols // 128, 128)
    bits = v.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    e = e.clamp(min=-22)
    q = (v * _pow2(-e).unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(rows, cols), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    if op in ("route", "train"):
        return _router_inputs(c, seed)
    g = _gen(seed)
    if op == "quant":
        dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        return dict(case=c, x=_activations(g, c["rows"], c["cols"], dtype))
    if op == "linear":
        x = _activations(g, c["M"], c["K"], torch.bfloat16)
        st = dict(case=c, w=_encode(_normal(g, (c["N"], c["K"]), 0.02), "ceil"))
        if c["act"] == "e2m1":
            st["x"] = x
        else:
            st["a"] = _e4m3_rows(x)
        return st
    if op == "step":
        return dict(case=c, x=_activations(g, c["T"], c["Cin"], torch.bfloat16),
                    w=_normal(g, (c["Cout"], c["Cin"]), 0.02, torch.bfloat16),
                    dy=_normal(g, (c["T"], c["Cout"]), 1e-3, torch.bfloat16))
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    like = torch.randn((1, E), generator=g, device=DEV)
    picked = (torch.randn((T, E), generator=g, device=DEV) + 0.5 * like).topk(k, 1).indices
    rows = torch.bincount(picked.reshape(-1), minlength=E).tolist()
    offs = [0]
    for r in rows:
        offs.append(offs[-1] + (r + 15) // 16 * 16)
    cap = T * k + 15 * E  # the bound that holds for every routing: rows past offs[E] are not touched
    x = _activations(g, cap, K, torch.bfloat16)
    at = torch.arange(cap, device=DEV)
    begin = torch.tensor(offs[:-1] + [cap], device=DEV)
    seg = torch.bucketize(at, torch.tensor(offs[1:], device=DEV), right=True)
    x[at - begin[seg] >= torch.tensor(rows + [0], device=DEV)[seg]] = 0  # the padding rows of each expert
    q, s = zip(*[_encode(_normal(g, (N, K), 0.02), "ceil") for _ in range(E)])
    return dict(case=c, a=_e4m3_rows(x), w=(torch.stack(q), torch.stack(s)), rows=offs,
                offsets=torch.tensor(offs, dtype=torch.int32, device=DEV),
                d=torch.zeros((cap, N), dtype=torch.bfloat16, device=DEV))


# ---- the plain forms ------------------------------------------------------------

def _pow2(e):
    """2^e for whole e >= -127, as float32."""
    return ((e.clamp(min=-126) + 127) << 23).view(torch.float32) * torch.where(e < -126, 0.5, 1.0)


def _encode(x, rule):
    """MXFP4 codes [rows, ceil32(cols) / 2] and scales [ceil(cols / 256), rows, 8] of x [rows, cols]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % 32))
    v = x.view(rows, -1, 32)
    bits = v.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 127 - 2
    if rule == "ceil":
        e = e + ((bits & 0x7FFFFF) > 0x400000).int()
    e = torch.where(bits < 0x00800000, torch.full_like(e, -127), e).clamp(min=-127)
    v = v * _pow2(-e).unsqueeze(2)
    a = v.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte()) | (torch.signbit(v).byte() << 3)
    code = code.view(rows, -1, 2)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 8))
    return code[..., 0] | (code[..., 1] << 4), s.view(rows, -1, 8).transpose(0, 1).contiguous()


def _decode(q, s):
    """The values of MXFP4 codes q [rows, cols / 2] with scales s, as float32 [rows, cols]."""
    rows = q.shape[0]
    code = torch.stack((q & 15, q >> 4), 2).view(rows, -1)
    v = torch.tensor(GRID + tuple(-g for g in GRID), device=q.device)[code.int()]
    e = s.transpose(0, 1).reshape(rows, -1)[:, : code.shape[1] // 32].int() - 127
    return (v.view(rows, -1, 32) * _pow2(e).unsqueeze(2)).view(rows, -1)


def _decode_e4m3(q, s):
    rows, cols = q.shape
    return (q.view(torch.float8_e4m3fn).float().view(rows, -1, 128) * _pow2(s.int() - 127).unsqueeze(2)).view(rows, cols)


def _router_plain(st):
    c = st["case"]
    z = st["logits"].float()
    T, E, k = c["T"], c["E"], c["k"]
    live = (z > -math.inf).any(1)
    if st["mask"] is not None:
        live = live & st["mask"]
    z = torch.where(live.unsqueeze(1), z, torch.full_like(z, -math.inf))
    top, idx = torch.sort(z, dim=1, descending=True, stable=True)  # equal logits: the lowest expert first
    top, idx = top[:, :k], idx[:, :k]
    on = top > -math.inf
    if c["score"] == "softmax":
        m = torch.where(live, z.amax(1), torch.zeros_like(z[:, 0])).unsqueeze(1)
        s = torch.exp(z - m)
        p = s / torch.where(live, s.sum(1), torch.ones_like(z[:, 0])).unsqueeze(1)
        s, slope = p, None
    else:
        s = 1 / (1 + torch.exp(-z))
        p = s / torch.where(live, s.sum(1), torch.ones_like(z[:, 0])).unsqueeze(1)
        slope = 1 - s
    w = torch.where(on, s.gather(1, idx), torch.zeros_like(top))
    share = w
    if c["renorm"]:
        share = w / torch.where(live, w.sum(1), torch.ones_like(w[:, 0])).unsqueeze(1)
    weights = st["scale"] * share
    n = live.sum()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=z.device)
    counts.scatter_add_(0, idx.reshape(-1), on.reshape(-1).int())
    counts[E] = n
    f = st["coef"] * E / (k * n.clamp(min=1).float() ** 2)
    loss = f * (counts[:E].float() * p.sum(0)).sum()
    picked = torch.where(on, idx, torch.full_like(idx, -1)).int()
    if c["op"] == "route":
        return picked, weights, counts
    g = st["dloss"] * f * counts[:E].float()
    dz = p * (g - (g * p).sum(1, keepdim=True))
    dw = torch.where(on, st["dweights"], torch.zeros_like(top)) * st["scale"]
    if c["score"] == "sigmoid":
        dz = dz * slope
        d = share * (dw - (dw * share).sum(1, keepdim=True)) if c["renorm"] else share * dw
        d = d * slope.gather(1, idx)
    elif c["renorm"]:
        d = share * (dw - (dw * share).sum(1, keepdim=True))
    else:
        d = share * dw
        dz = dz - p * d.sum(1, keepdim=True)
    dz = dz.scatter_add(1, idx, torch.where(on, d, torch.zeros_like(d)))
    return picked, weights, counts, loss, dz.to(st["logits"].dtype)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op in ("route", "train"):
        return _router_plain(st)
    if op == "quant":
        out = [_decode(*_encode(st["x"], c["rule"])).bfloat16()]
        if c["both"]:
            out.append(_decode(*_encode(st["x"].t(), c["rule"])).bfloat16())
        return out
    if op == "linear":
        a = _decode(*_encode(st["x"], "ceil")) if c["act"] == "e2m1" else _decode_e4m3(*st["a"])
        y = a @ _decode(*st["w"]).t()
        return y.bfloat16() if c["out"] == "bf16" else y
    if op == "step":
        x, w, dy = st["x"], st["w"], st["dy"]
        y = _decode(*_encode(x, "ceil")) @ _decode(*_encode(w, "ceil")).t()
        dx = _decode(*_encode(dy, "ceil")) @ _decode(*_encode(w.t(), "ceil")).t()
        dw = _decode(*_encode(dy.t(), "ceil")) @ _decode(*_encode(x.t(), "ceil")).t()
        return y.bfloat16(), dx.bfloat16(), dw
    a = _decode_e4m3(*st["a"])
    q, s = st["w"]
    d = st["d"]
    for e, (lo, hi) in enumerate(zip(st["rows"], st["rows"][1:])):
        if hi > lo:
            d[lo:hi] = (a[lo:hi] @ _decode(q[e], s[e]).t()).bfloat16()
    return d


# ---- the framework's operators ----------------------------------------------------

def _own(st):
    import fine_grained_blockwise_amd as fgb

    c = st["case"]
    op = c["op"]
    if op in ("route", "train"):
        how = dict(score=fgb.ROUTER_SOFTMAX if c["score"] == "softmax" else fgb.ROUTER_SIGMOID, renorm=c["renorm"],
                   scale=st["scale"])
        if op == "route":
            return fgb.moe_router(st["logits"], c["k"], token_mask=st["mask"], **how)[:3]
        how["loss_coef"] = st["coef"]
        idx, weights, counts, loss = fgb.moe_router(st["logits"], c["k"], token_mask=st["mask"], **how)
        dz = fgb.moe_router_backward(st["logits"], idx, counts, st["dweights"], st["dloss"], **how)
        return idx, weights, counts, loss, dz
    if op == "quant":
        rule = fgb.SCALE_CEIL if c["rule"] == "ceil" else fgb.SCALE_OCP_FLOOR
        if not c["both"]:
            return [fgb.mxfp4_dequant(*fgb.mxfp4_quant(st["x"], rule=rule), out_dtype=torch.bfloat16)]
        q, s, qt, s_t = fgb.mxfp4_quant_t(st["x"], rule=rule)
        return [fgb.mxfp4_dequant(q, s, out_dtype=torch.bfloat16), fgb.mxfp4_dequant(qt, s_t, out_dtype=torch.bfloat16)]
    if op == "linear":
        out = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        if c["act"] == "e2m1":
            return fgb.mxfp4_gemm(*fgb.mxfp4_quant(st["x"]), *st["w"], out_dtype=out)
        return fgb.mxfp4_gemm(*st["a"], *st["w"], a_fmt=fgb.E4M3, out_dtype=out)
    if op == "step":
        xq, xs, xqt, xst = fgb.mxfp4_quant_t(st["x"])
        wq, ws, wqt, wst = fgb.mxfp4_quant_t(st["w"])
        gq, gs, gqt, gst = fgb.mxfp4_quant_t(st["dy"])
        return (fgb.mxfp4_gemm(xq, xs, wq, ws), fgb.mxfp4_gemm(gq, gs, wqt, wst),
                fgb.mxfp4_gemm(gqt, gst, xqt, xst, out_dtype=torch.float32))
    return fgb.mxfp4_grouped_gemm(*st["a"], *st["w"], st["offsets"], a_fmt=fgb.E4M3, d=st["d"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    c = case
    op = c["op"]
    fp4 = 17 / 32  # bytes of an element: half a byte, and a thirty-second of its group's scale
    if op in ("route", "train"):
        T, E, k = c["T"], c["E"], c["k"]
        z = T * E * (4 if c["dtype"] == "f32" else 2)
        fwd = z + 8 * T * k + (T if c["masked"] else 0) + 4 * E
        if op == "route":
            return dict(bytes=fwd, flops=4 * T * E)
        return dict(bytes=fwd + 2 * z + 8 * T * k, flops=12 * T * E)
    if op == "quant":
        n = c["rows"] * c["cols"]
        each = n * (2 * fp4 + 2)
        return dict(bytes=n * (4 if c["dtype"] == "f32" else 2) + each * (2 if c["both"] else 1), flops=4 * n)
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        a = 2 if c["act"] == "e2m1" else 1 + 1 / 128
        return dict(bytes=M * K * a + N * K * fp4 + M * N * (2 if c["out"] == "bf16" else 4), flops=2 * M * N * K)
    if op == "step":
        T, I, O = c["T"], c["Cin"], c["Cout"]
        return dict(bytes=2 * (T * I + I * O + T * O) + 2 * T * O + 2 * T * I + 4 * I * O, flops=6 * T * I * O)
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    busy = E * (1 - (1 - k / E) ** T)
    return dict(bytes=busy * N * K * fp4 + T * k * (K + 2 * N), flops=2 * T * k * N * K)


# ---- the same from the definitions, in 64 bits ------------------------------------------

def _two_to(e):
    """2^e as float64, built from its bits (pow() may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(x, rule, biggest=6.0, emax=2, lowest=-127, group=32):
    """x [rows, cols] on the grid of its groups: each element is the nearest multiple of its binade's step (ties
    to the even multiple) after division by 2^e, e the group's exponent."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -cols % group)).view(rows, -1, group)
    most = x.abs().amax(2, keepdim=True)
    mant, ex = torch.frexp(most)                 # most = mant 2^ex, mant in [1/2, 1)
    e = ex.double() - 1 - emax
    if rule == "ceil":
        e = e + (mant * 2 > biggest / 2 ** emax).double()
    e = torch.where(most > 0, e, torch.full_like(e, lowest)).clamp(min=lowest)
    y = x * _two_to(-e)
    binade = torch.frexp(y)[1].double().clamp(min=1) - 1           # [1, 2) and below share the step 1/2
    step = _two_to(binade - 1)
    y = (torch.round(y / step) * step).clamp(-biggest, biggest)     # round(): ties to even
    return (y * _two_to(e)).view(rows, -1)


def _exact_decode(q, s):
    rows, half = q.shape
    code = torch.empty((rows, 2 * half), dtype=torch.uint8, device=q.device)
    code[:, 0::2], code[:, 1::2] = q % 16, q // 16
    ex, man = (code >> 1) & 3, (code & 1).double() / 2
    v = torch.where(ex == 0, man, (1 + man) * _two_to(ex.long() - 1)) * (1 - 2 * (code >> 3).double())
    at = torch.arange(2 * half, device=q.device)
    sc = s[at // 256, :, at // 32 % 8].t()
    return v * _two_to(sc.long() - 127)


def _exact_e4m3(q, s):
    c = q.int()
    ex, man = (c >> 3) & 15, (c & 7).double() / 8
    v = torch.where(ex == 0, man * 2.0 ** -6, (1 + man) * _two_to(ex - 7)) * (1 - 2 * (c >> 7)).double()
    return v * _two_to(s.long() - 127).repeat_interleave(128, 1)


def _exact_router(st):
    c = st["case"]
    E, k = c["E"], c["k"]
    z = st["logits"].double().cpu().numpy()
    use = np.ones(len(z), bool) if st["mask"] is None else st["mask"].cpu().numpy()
    live = use & np.isfinite(z).any(1)
    order = np.argsort(-z, 1, kind="stable")[:, :k]
    on = live[:, None] & np.isfinite(np.take_along_axis(z, order, 1))
    with np.errstate(all="ignore"):
        if c["score"] == "softmax":
            s = np.exp(z - z.max(1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
        else:
            s = 1 / (1 + np.exp(-z))
        s[~live] = 0
        total = np.where(live, s.sum(1), 1)[:, None]
        p = s / total
    chosen = np.where(on, np.take_along_axis(s, order, 1), 0)
    norm = np.where(live, chosen.sum(1), 1)[:, None] if c["renorm"] else np.ones((len(z), 1))
    counts = np.bincount(order[on], minlength=E)
    n = int(live.sum())
    f = st["coef"] * E / (k * max(n, 1) ** 2)
    loss = f * (counts * p.sum(0)).sum()
    out = [torch.from_numpy(np.where(on, order, -1).astype(np.int32)), torch.from_numpy(st["scale"] * chosen / norm),
           torch.from_numpy(np.append(counts, n).astype(np.int32))]
    if c["op"] == "route":
        return out
    # through the scores: d(loss + sum dw weights) / ds, then ds/dz
    dw = np.where(on, st["dweights"].double().cpu().numpy(), 0) * st["scale"]
    gp = float(st["dloss"]) * f * counts
    ds = (gp - (gp * p).sum(1, keepdims=True)) / total
    dc = (dw - ((dw * chosen).sum(1, keepdims=True) / norm if c["renorm"] else 0)) / norm
    full = np.zeros_like(z)
    np.put_along_axis(full, order, np.where(on, dc, 0), 1)
    ds = np.where(live[:, None], ds + full, 0)
    dz = s * (ds - (ds * s).sum(1, keepdims=True)) if c["score"] == "softmax" else s * (1 - s) * ds
    return out + [torch.tensor(loss), torch.from_numpy(dz)]


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    op = c["op"]
    if op in ("route", "train"):
        return _exact_router(st)
    if op == "quant":
        out = [_exact_values(st["x"], c["rule"])]
        if c["both"]:
            out.append(_exact_values(st["x"].t(), c["rule"]))
        return out
    if op == "linear":
        a = _exact_values(st["x"], "ceil") if c["act"] == "e2m1" else _exact_e4m3(*st["a"])
        return a @ _exact_decode(*st["w"]).t()
    if op == "step":
        x, w, dy = st["x"], st["w"], st["dy"]
        return (_exact_values(x, "ceil") @ _exact_values(w, "ceil").t(),
                _exact_values(dy, "ceil") @ _exact_values(w.t(), "ceil").t(),
                _exact_values(dy.t(), "ceil") @ _exact_values(x.t(), "ceil").t())
    a = _exact_e4m3(*st["a"])
    d = torch.zeros((a.shape[0], c["N"]), dtype=torch.float64, device=DEV)
    for e, (lo, hi) in enumerate(zip(st["rows"], st["rows"][1:])):
        if hi > lo:
            d[lo:hi] = a[lo:hi] @ _exact_decode(st["w"][0][e], st["w"][1][e]).t()
    return d
