"""Cases of the norm before an FP8 product, of the router with a bias and groups, and of gradient clipping, for timing
and comparison.

Every case names an operation and its sizes:

  norm       RMSNorm with the residual's addition, into E4M3 codes with power-of-two scales: returns the values that
             codes and scales stand for, the new residual stream, 1 / rms of each row, and (y = True) the norm itself
  norm_grad  its gradient: of the residual stream (that of the stream behind it added) and of the weight
  route      the router's forward pass (serving) with a bias for balance and the choice limited to groups of experts:
             the experts of each token, their weights, the slots per expert
  train      the router's forward and backward pass: the balance loss, the gradient of the logits, the next bias
  clip       the global norm of many gradients, and the clipped gradients in the type that the optimiser takes

A case's types are "f32" and "bf16".
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one token's hidden state in a decode step
        dict(name="norm_token", op="norm", rows=1, cols=7168, x="bf16", stream="bf16", w="bf16", residual=True,
             group=128, y=False),
        # a prompt of odd length, an FP32 residual stream, scales of 32 columns, the norm kept for the router
        dict(name="norm_odd_f32", op="norm", rows=1009, cols=2080, x="bf16", stream="f32", w="f32", residual=True,
             group=32, y=True),
        # a training batch
        dict(name="norm_8k", op="norm", rows=8192, cols=7168, x="bf16", stream="bf16", w="bf16", residual=True,
             group=128, y=False),
        # the gradient for an odd number of tokens and an FP32 stream
        dict(name="grad_odd_f32", op="norm_grad", rows=1009, cols=2080, dy="bf16", stream="f32", w="f32",
             residual=True),
        # the gradient for a training batch
        dict(name="grad_8k", op="norm_grad", rows=8192, cols=7168, dy="bf16", stream="bf16", w="bf16", residual=True),
        # one token of a decode step, four of eight groups
        dict(name="route_token", op="route", T=1, E=256, k=8, G=8, kg=4, score="sigmoid", bias=True, renorm=True,
             dtype="f32", masked=False),
        # a ragged batch with padding tokens and disabled experts, groups that are no power of two, bf16 logits
        dict(name="route_odd", op="route", T=4999, E=160, k=6, G=8, kg=3, score="softmax", bias=False, renorm=False,
             dtype="bf16", masked=True),
        # many experts without groups, a bias alone
        dict(name="train_bias_e384", op="train", T=2047, E=384, k=8, G=1, kg=1, score="sigmoid", bias=True,
             renorm=True, dtype="bf16", masked=False),
        # a training batch, four of eight groups
        dict(name="train_16k_e256", op="train", T=16384, E=256, k=8, G=8, kg=4, score="sigmoid", bias=True,
             renorm=True, dtype="f32", masked=False),
        # the weights of a model's norms: many small gradients
        dict(name="clip_norms", op="clip", n=122, low=7168, high=7168, f32=0.0, out="f32", clipped=True),
        # gradients of all sizes, in both types, of lengths that no vector divides, none above the limit
        dict(name="clip_ragged", op="clip", n=301, low=1, high=4000000, f32=0.5, out="bf16", clipped=False),
        # the FP32 weight gradients of 32 experts' products, an expert's apart
        dict(name="clip_experts", op="clip", n=64, low=14680064, high=29360128, f32=1.0, out="bf16", clipped=True),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return step * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_grad", "route", "train", "clip"])
    types = ["f32", "bf16"]
    if op == "norm":
        group = rng.choice([32, 128])
        return dict(op=op, rows=log(1, 8192), cols=log(1, 7168 // group, group), x=rng.choice(types),
                    stream=rng.choice(types), w=rng.choice(types), residual=rng.random() < 0.7, group=group,
                    y=rng.random() < 0.5)
    if op == "norm_grad":
        return dict(op=op, rows=log(1, 8192), cols=log(1, 224, 32), dy=rng.choice(types), stream=rng.choice(types),
                    w=rng.choice(types), residual=rng.random() < 0.7)
    if op == "clip":
        low = log(1, 100000)
        return dict(op=op, n=log(1, 400), low=low, high=low * rng.randint(1, 40), f32=rng.choice([0.0, 0.3, 1.0]),
                    out=rng.choice(types), clipped=rng.random() < 0.6)
    G = rng.choice([1, 2, 3, 4, 8, 16])
    size = log(2, 64 if G > 4 else 128)
    kg = rng.randint(1, G)
    k = rng.randint(1, min(8, kg * size))
    return dict(op=op, T=log(1, 16384), E=min(G * size, 1024 // G * G), k=k, G=G, kg=kg,
                score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, renorm=rng.random() < 0.6,
                dtype=rng.choice(types), masked=rng.random() < 0.4)


# ---- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _hidden(g, rows, cols, dtype, std):
    # hidden states: tokens of different size, a few channels much larger than the rest
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= std * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    big = torch.rand((cols,), generator=g, device=DEV) < 0.01
    return torch.where(big, 20.0 * x, x).to(dtype)


def _router_inputs(c, g):
    T, E = c["T"], c["E"]
    skew = torch.randn((1, E), generator=g, device=DEV)  # some experts are liked more
    z = 1.5 * torch.randn((T, E), generator=g, device=DEV) + skew
    st = dict(case=c, mask=None, bias=None, scale=2.5 if c["score"] == "sigmoid" else 1.0, coef=0.01, rate=1e-3)
    if c["masked"]:
        z[torch.rand((T, E), generator=g, device=DEV) < 0.1] = -math.inf      # experts a token may not use
        z[torch.rand((T,), generator=g, device=DEV) < 0.02] = -math.inf       # tokens with none left
        st["mask"] = torch.rand((T,), generator=g, device=DEV) < 0.9          # padding tokens
    if c["bias"]:  # what the updates have come to: against the skew
        st["bias"] = (-0.1 * skew + 0.02 * torch.randn((1, E), generator=g, device=DEV)).view(E)
    st["logits"] = z.to(TYPES[c["dtype"]])
    if c["op"] == "train":
        st["dweights"] = 1e-2 * torch.randn((T, c["k"]), generator=g, device=DEV)
        st["dloss"] = torch.ones((), device=DEV)
    return st


def _clip_inputs(c, g):
    pick = np.random.default_rng(c["n"])  # the model's tensors: the same for every seed
    n, low, high = c["n"], c["low"], c["high"]
    if low * 2 == high:  # two matrices an expert
        sizes = [low, high] * (n // 2) + [low] * (n % 2)
    else:
        sizes = [int(v) for v in np.exp(pick.uniform(math.log(low), math.log(high), n)).round()]
    kinds = [torch.float32 if v < c["f32"] else torch.bfloat16 for v in pick.random(n)]
    grads = [(torch.randn((s,), generator=g, device=DEV) * v).to(t)
             for s, t, v in zip(sizes, kinds, np.exp(pick.normal(-7, 1, n)).tolist())]
    # the clipped gradients: slices of one bucket, each at a multiple of 64 elements
    starts = np.concatenate([[0], np.cumsum([(s + 63) // 64 * 64 for s in sizes])]).tolist()
    bucket = torch.zeros((starts[-1],), dtype=TYPES[c["out"]], device=DEV)
    outs = [bucket[a: a + s] for a, s in zip(starts, sizes)]
    typical = math.exp(-7 + 0.5) * math.sqrt(sum(sizes))
    return dict(case=c, grads=grads, outs=outs, bucket=bucket, starts=starts, scale=0.25,
                max_norm=0.25 * typical * (0.1 if c["clipped"] else 100.0))


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    if c["op"] in ("route", "train"):
        return _router_inputs(c, g)
    if c["op"] == "clip":
        return _clip_inputs(c, g)
    rows, cols = c["rows"], c["cols"]
    stream = TYPES[c["stream"]]
    w = (1.0 + 0.2 * torch.randn((cols,), generator=g, device=DEV)).to(TYPES[c["w"]])
    st = dict(case=c, w=w)
    if c["op"] == "norm":
        st["x"] = _hidden(g, rows, cols, TYPES[c["x"]], 0.5)
        st["r"] = _hidden(g, rows, cols, stream, 2.0) if c["residual"] else None
        return st
    st["h"] = _hidden(g, rows, cols, stream, 2.0)
    st["rstd"] = torch.rsqrt(st["h"].double().square().mean(1) + EPS).float()
    st["dy"] = (1e-3 * torch.randn((rows, cols), generator=g, device=DEV)).to(TYPES[c["dy"]])
    st["dh"] = (1e-3 * torch.randn((rows, cols), generator=g, device=DEV)).to(stream) if c["residual"] else None
    return st


# ---- the plain forms ------------------------------------------------------------

def _pow2(e):
    """2^e for whole e >= -127, as float32."""
    return ((e.clamp(min=-126) + 127) << 23).view(torch.float32) * torch.where(e < -126, 0.5, 1.0)


def _norm_plain(st):
    c = st["case"]
    rows, cols, group = c["rows"], c["cols"], c["group"]
    h = st["x"] if st["r"] is None else (st["x"].float() + st["r"].float()).to(st["r"].dtype)
    f = h.float()
    rstd = 1 / torch.sqrt(f.square().mean(1) + EPS)
    y = f * rstd.unsqueeze(1) * st["w"].float()
    v = y.view(rows, cols // group, group)
    bits = v.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    low = -22 if group == 128 else -127
    e = torch.where(bits < 0x00800000, torch.full_like(e, low), e).clamp(min=low).unsqueeze(2)
    q = (v * _pow2(-e)).to(torch.float8_e4m3fn)
    out = dict(values=(q.float() * _pow2(e)).view(rows, cols).bfloat16(), rstd=rstd)
    if st["r"] is not None:
        out["h"] = h
    if c["y"]:
        out["y"] = y.bfloat16()
    return out


def _norm_grad_plain(st):
    rstd = st["rstd"].unsqueeze(1)
    hat = st["h"].float() * rstd
    dy = st["dy"].float()
    a = dy * st["w"].float()
    dx = rstd * (a - hat * (a * hat).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return dx.to(st["h"].dtype), (dy * hat).sum(0)


def _router_plain(st):
    c = st["case"]
    z = st["logits"].float()
    T, E, k, G, kg = (c[n] for n in ("T", "E", "k", "G", "kg"))
    none = torch.full_like(z, -math.inf)
    if st["mask"] is not None:
        z = torch.where(st["mask"].unsqueeze(1), z, none)
    usable = z > -math.inf
    live = usable.any(1)
    one = torch.ones_like(z[:, 0])
    # the scores in 64 bits, rounded once: the choice compares values that may differ by a rounding only
    d = z.double()
    if c["score"] == "softmax":
        t = torch.exp(d - torch.where(live, d.amax(1), torch.zeros_like(d[:, 0])).unsqueeze(1))
        s = (t / torch.where(live, t.sum(1), torch.ones_like(t[:, 0])).unsqueeze(1)).float()
        p, slope = s, None
    else:
        s = (1 / (1 + torch.exp(-d))).float()
        p = s / torch.where(live, s.sum(1), one).unsqueeze(1)
        slope = 1 - s
    value = z if st["bias"] is None else torch.where(usable, s + st["bias"], none)
    if G > 1:
        best = torch.sort(value.view(T, G, E // G), dim=2, descending=True)[0][:, :, :2]
        has = best[:, :, 0] > -math.inf
        of = best[:, :, 0]
        if st["bias"] is not None:
            of = torch.where(has, torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2), of)
        order = torch.sort(of, dim=1, descending=True, stable=True)[1][:, :kg]  # equal groups: the lowest first
        open_ = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, order, True)
        value = torch.where(open_.repeat_interleave(E // G, 1), value, none)
    top, idx = torch.sort(value, dim=1, descending=True, stable=True)  # equal values: the lowest expert first
    top, idx = top[:, :k], idx[:, :k]
    on = top > -math.inf
    w = torch.where(on, s.gather(1, idx), torch.zeros_like(top))
    share = w / torch.where(live, w.sum(1), one).unsqueeze(1) if c["renorm"] else w
    weights = st["scale"] * share
    n = live.sum()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=z.device)
    counts.scatter_add_(0, idx.reshape(-1), on.reshape(-1).int())
    counts[E] = n
    picked = torch.where(on, idx, torch.full_like(idx, -1)).int()
    if c["op"] == "route":
        return picked, weights, counts
    f = st["coef"] * E / (k * n.clamp(min=1).float() ** 2)
    loss = f * (counts[:E].double() * p.double().sum(0)).sum()
    g = st["dloss"] * f * counts[:E].float()
    dz = p * (g - (g * p).sum(1, keepdim=True))
    dw = torch.where(on, st["dweights"], torch.zeros_like(top)) * st["scale"]
    own_part = share * (dw - (dw * share).sum(1, keepdim=True)) if c["renorm"] else share * dw
    if c["score"] == "sigmoid":
        dz = dz * slope
        own_part = own_part * slope.gather(1, idx)
    elif not c["renorm"]:
        dz = dz - p * own_part.sum(1, keepdim=True)
    dz = dz.scatter_add(1, idx, torch.where(on, own_part, torch.zeros_like(own_part)))
    out = [picked, weights, counts, loss.float(), dz.to(st["logits"].dtype)]
    if st["bias"] is not None:
        mean = counts[:E].double().mean()
        out.append(st["bias"] + st["rate"] * torch.sign(mean - counts[:E]).float())
    return out


def _clip_plain(st):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum()
    norm = st["scale"] * torch.sqrt(total)
    factor = (st["scale"] * torch.clamp(st["max_norm"] / norm, max=1.0)).float()
    [o.copy_(g.float() * factor) for o, g in zip(st["outs"], st["grads"])]
    return norm.float(), st["bucket"]


PLAIN = dict(norm=_norm_plain, norm_grad=_norm_grad_plain, route=_router_plain, train=_router_plain, clip=_clip_plain)


# ---- the framework's operators ----------------------------------------------------

def _own(st):
    import fine_grained_blockwise_amd as fgb

    c = st["case"]
    op = c["op"]
    if op == "norm":
        q, s, y, h, rstd = fgb.rmsnorm_quant(st["x"], st["w"], residual=st["r"], eps=EPS, group=c["group"],
                                             y_dtype=torch.bfloat16 if c["y"] else None)
        out = dict(values=fgb.fp8_dequant(q, s, fgb.ROW1x128 if c["group"] == 128 else fgb.ROW1x32, torch.bfloat16),
                   rstd=rstd)
        if st["r"] is not None:
            out["h"] = h
        if c["y"]:
            out["y"] = y
        return out
    if op == "norm_grad":
        return fgb.rmsnorm_backward(st["dy"], st["h"], st["w"], st["rstd"], dh=st["dh"])
    if op == "clip":
        return fgb.grad_clip(st["grads"], st["max_norm"], scale=st["scale"], out=st["outs"]), st["bucket"]
    how = dict(score=fgb.ROUTER_SOFTMAX if c["score"] == "softmax" else fgb.ROUTER_SIGMOID, renorm=c["renorm"],
               scale=st["scale"])
    choice = dict(token_mask=st["mask"], bias=st["bias"], groups=c["G"], topk_groups=c["kg"])
    if op == "route":
        return fgb.moe_router(st["logits"], c["k"], **how, **choice)[:3]
    how["loss_coef"] = st["coef"]
    idx, weights, counts, loss = fgb.moe_router(st["logits"], c["k"], **how, **choice)
    dz = fgb.moe_router_backward(st["logits"], idx, counts, st["dweights"], st["dloss"], **how)
    out = [idx, weights, counts, loss, dz]
    if st["bias"] is not None:
        out.append(fgb.moe_bias_update(st["bias"], counts, st["rate"]))
    return out


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    c = case
    op = c["op"]
    size = dict(f32=4, bf16=2)
    if op in ("norm", "norm_grad"):
        n = c["rows"] * c["cols"]
        stream = size[c["stream"]]
        if op == "norm":
            # the codes and scales written and read again, their values written
            each = size[c["x"]] + 2 * (1 + 1 / c["group"]) + 2 + (2 * stream if c["residual"] else 0) + (2 if c["y"] else 0)
            return dict(bytes=n * each + 4 * c["rows"] + size[c["w"]] * c["cols"], flops=8 * n)
        each = size[c["dy"]] + 2 * stream + (stream if c["residual"] else 0)
        return dict(bytes=n * each + 4 * c["rows"] + (size[c["w"]] + 4) * c["cols"], flops=12 * n)
    if op in ("route", "train"):
        T, E, k = c["T"], c["E"], c["k"]
        z = T * E * size[c["dtype"]]
        fwd = z + 8 * T * k + (T if c["masked"] else 0) + 4 * E + (4 * E if c["bias"] else 0)
        if op == "route":
            return dict(bytes=fwd, flops=6 * T * E)
        return dict(bytes=fwd + 2 * z + 8 * T * k, flops=14 * T * E)
    if c["low"] * 2 == c["high"]:
        n = c["n"] * (c["low"] + c["high"]) / 2
    elif c["low"] == c["high"]:
        n = c["n"] * c["low"]
    else:
        n = c["n"] * (c["high"] - c["low"]) / math.log(c["high"] / c["low"])  # the mean of the lengths drawn
    return dict(bytes=n * (4 * c["f32"] + 2 * (1 - c["f32"]) + size[c["out"]]), flops=3 * n)


# ---- the same from the definitions, in 64 bits ------------------------------------------

def _two_to(e):
    """2^e as float64, built from its bits (pow() may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(y, group):
    """y [rows, cols] on the grid of its groups: the nearest multiple of its binade's step (ties to the even multiple)
    after division by 2^e, e the group's exponent."""
    rows, cols = y.shape
    y = y.view(rows, -1, group)
    most = y.abs().amax(2, keepdim=True)
    mant, ex = torch.frexp(most)                 # most = mant 2^ex, mant in [1/2, 1)
    low = -22 if group == 128 else -127
    e = ex.double() - 9 + (mant > 0.875).double()
    e = torch.where(most > 0, e, torch.full_like(e, low)).clamp(min=low)
    v = y * _two_to(-e)
    step = _two_to(torch.frexp(v)[1].double().clamp(min=-5) - 4)     # three bits behind the first, 2^-9 at least
    v = (torch.round(v / step) * step).clamp(-448, 448)              # round(): ties to even
    return (v * _two_to(e)).view(rows, cols)


def _exact_router(st):
    c = st["case"]
    T, E, k, G, kg = (c[n] for n in ("T", "E", "k", "G", "kg"))
    z = st["logits"].double().cpu().numpy()
    if st["mask"] is not None:
        z[~st["mask"].cpu().numpy()] = -np.inf
    live = np.isfinite(z).any(1)
    with np.errstate(all="ignore"):
        if c["score"] == "softmax":
            s = np.exp(z - z.max(1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
        else:
            s = 1 / (1 + np.exp(-z))
    s[~live] = 0
    total = np.where(live, s.sum(1), 1)[:, None]
    p = s / total
    value = z
    if st["bias"] is not None:  # by the definition both the score and its sum with the bias are FP32 numbers
        value = np.where(np.isfinite(z), s.astype(np.float32) + st["bias"].cpu().numpy(), np.float32(-np.inf))
    if G > 1:
        part = -np.sort(-value.reshape(T, G, E // G), 2)
        of = part[:, :, 0]
        if st["bias"] is not None:
            second = part[:, :, 1]
            of = of + np.where(np.isfinite(second), second, np.float32(0))
        order = np.argsort(-of, 1, kind="stable")[:, :kg]
        shut = np.ones((T, G), bool)
        np.put_along_axis(shut, order, False, 1)
        value = np.where(np.repeat(shut, E // G, 1), -np.inf, value)
    order = np.argsort(-value, 1, kind="stable")[:, :k]
    on = np.isfinite(np.take_along_axis(value, order, 1))
    chosen = np.where(on, np.take_along_axis(s, order, 1), 0)
    norm = np.where(live, chosen.sum(1), 1)[:, None] if c["renorm"] else np.ones((T, 1))
    counts = np.bincount(order[on], minlength=E)
    n = int(live.sum())
    out = [torch.from_numpy(np.where(on, order, -1).astype(np.int32)), torch.from_numpy(st["scale"] * chosen / norm),
           torch.from_numpy(np.append(counts, n).astype(np.int32))]
    if c["op"] == "route":
        return out
    f = st["coef"] * E / (k * max(n, 1) ** 2)
    # through the scores: d(loss + sum dw weights) / ds, then ds/dz
    dw = np.where(on, st["dweights"].double().cpu().numpy(), 0) * st["scale"]
    gp = float(st["dloss"]) * f * counts
    ds = (gp - (gp * p).sum(1, keepdims=True)) / total
    dc = (dw - ((dw * chosen).sum(1, keepdims=True) / norm if c["renorm"] else 0)) / norm
    full = np.zeros_like(z)
    np.put_along_axis(full, order, np.where(on, dc, 0), 1)
    ds = np.where(live[:, None], ds + full, 0)
    dz = s * (ds - (ds * s).sum(1, keepdims=True)) if c["score"] == "softmax" else s * (1 - s) * ds
    out += [torch.tensor(f * (counts * p.sum(0)).sum()), torch.from_numpy(dz)]
    if st["bias"] is not None:
        out.append(torch.from_numpy(st["bias"].double().cpu().numpy() + st["rate"] * np.sign(counts.mean() - counts)))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    op = c["op"]
    if op in ("route", "train"):
        return _exact_router(st)
    if op == "clip":
        total = math.fsum(float((g.double() ** 2).sum()) for g in st["grads"])
        norm = st["scale"] * math.sqrt(total)
        factor = st["scale"] * min(1.0, st["max_norm"] / norm)
        bucket = torch.zeros(st["bucket"].shape, dtype=torch.float64, device=DEV)
        for a, g in zip(st["starts"], st["grads"]):
            bucket[a: a + g.numel()] = g.double() * factor
        return torch.tensor(norm, dtype=torch.float64), bucket
    w = st["w"].double()
    if op == "norm":
        h = st["x"]
        if st["r"] is not None:  # the norm is that of the stream as it is stored
            h = (st["x"].double() + st["r"].double()).float().to(st["r"].dtype)
        rstd = (h.double().pow(2).sum(1) / c["cols"] + EPS) ** -0.5
        y = h.double() * rstd[:, None] * w
        out = dict(values=_exact_e4m3(y, c["group"]), rstd=rstd)
        if st["r"] is not None:
            out["h"] = h.double()
        if c["y"]:
            out["y"] = y
        return out
    # the Jacobian of h -> y row by row: rstd (I - hat hat^T / cols) applied to the weighted gradient
    hat = st["h"].double() * st["rstd"].double()[:, None]
    dy = st["dy"].double()
    inner = torch.einsum("rc,rc,c->r", hat, dy, w) / c["cols"]
    dx = st["rstd"].double()[:, None] * (dy * w - inner[:, None] * hat)
    if st["dh"] is not None:
        dx = dx + st["dh"].double()
    return dx, (dy * hat).sum(0)
