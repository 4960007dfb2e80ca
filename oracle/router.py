"""The MoE router and its gradient in numpy and 64 bits (TEST INFRASTRUCTURE)."""
import numpy as np

SOFTMAX, SIGMOID = 0, 1


def select(z, k, mask=None):
    """Ids [T, k] of the k largest logits (ties: lowest id; -inf and NaN never; -1 left over)."""
    T, E = z.shape
    key = np.where(np.isnan(z), -np.inf, z)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ok = np.take_along_axis(key, idx, 1) > -np.inf
    if mask is not None:
        ok &= np.asarray(mask, bool)[:, None]
    return np.where(ok, idx, -1).astype(np.int32)


def choose(z, k, score=SOFTMAX, bias=None, groups=1, topk_groups=1, mask=None):
    """Ids [T, k] where a bias and groups decide: the k largest c (ties: lowest id) in the topk_groups groups of
    largest value.  c = FP32(FP32(s) + bias), or the logits without a bias."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    c = np.where(z > -np.inf, z, -np.inf)  # NaN too
    if bias is not None:
        for t in range(T):
            ok = c[t] > -np.inf
            with np.errstate(all="ignore"):
                if score == SOFTMAX:
                    top = z[t, ok].max(initial=-np.inf)
                    s = np.where(z[t, ok] == top, 1.0, np.exp(z[t, ok] - top))
                    s = s / s.sum() if s.size else s
                else:
                    s = 1 / (1 + np.exp(-z[t, ok]))
                v = s.astype(np.float32) + np.asarray(bias, np.float32)[ok]
            c[t, ok] = np.where(np.isnan(v), -np.inf, v)
    if groups > 1:
        part = -np.sort(-c.reshape(T, groups, E // groups), axis=2)
        value = part[:, :, 0].copy()
        if bias is not None and E // groups > 1:
            second = part[:, :, 1]
            with np.errstate(all="ignore"):
                both = value.astype(np.float32) + second.astype(np.float32)
            value = np.where(second > -np.inf, both, value)
        # (a group with nothing to choose after one whose sum of two is -inf)
        best = np.lexsort((-value, part[:, :, 0] == -np.inf), axis=1)[:, :topk_groups]
        shut = np.ones((T, groups), bool)
        np.put_along_axis(shut, best, False, 1)
        c = np.where(np.repeat(shut, E // groups, 1), -np.inf, c)
    return select(c, k, mask)


def scores(z, score):
    """(s, p) of rows with at least one usable logit."""
    with np.errstate(all="ignore"):
        if score == SOFTMAX:
            s = np.exp(z - np.nanmax(z, 1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
            return s, s
        s = np.where(z > 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        return s, np.exp(log_sigmoid(z) - log_sigmoid(z).max(1, keepdims=True)) / np.exp(
            log_sigmoid(z) - log_sigmoid(z).max(1, keepdims=True)).sum(1, keepdims=True)


def log_sigmoid(z):
    with np.errstate(all="ignore"):
        return np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))


def forward(z, k, score=SOFTMAX, renorm=False, scale=1.0, coef=0.0, mask=None, idx=None):
    """-> dict(idx, weights, counts [E + 1], loss); idx: the choice, where it is not select()'s."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    idx = select(z, k, mask) if idx is None else idx
    live = (idx >= 0).any(1)
    weights, psum = np.zeros((T, k)), np.zeros(E)
    for t in np.flatnonzero(live):
        s, p = (v[0] for v in scores(z[t:t + 1], score))
        on = idx[t] >= 0
        if renorm:
            l = z[t, idx[t, on]] if score == SOFTMAX else log_sigmoid(z[t, idx[t, on]])
            r = np.exp(l - l.max())
            weights[t, on] = scale * r / r.sum()
            if np.isnan(p).any():
                weights[t, on] = np.nan
        else:
            weights[t, on] = scale * s[idx[t, on]]
        psum += p
    counts = np.bincount(idx[idx >= 0], minlength=E)
    n = int(live.sum())
    loss = coef * E / (k * max(n, 1) ** 2) * float((counts * psum).sum())
    return dict(idx=idx, weights=weights, counts=np.append(counts, n).astype(np.int32), loss=loss)


def objective(z, idx, counts, dweights, dloss, score, renorm, scale, coef):
    """sum dweights * weights + dloss * loss as a function of z alone, the choices and counts held fixed: what the
    gradient differentiates."""
    T, E = z.shape
    k = idx.shape[1]
    n = max(int(counts[E]), 1)
    total = 0.0
    for t in range(T):
        on = idx[t] >= 0
        if not on.any():
            continue
        s, p = (v[0] for v in scores(z[t:t + 1], score))
        w = s[idx[t, on]]
        if renorm:
            l = z[t, idx[t, on]] if score == SOFTMAX else log_sigmoid(z[t, idx[t, on]])
            w = np.exp(l - l.max())
            w = w / w.sum()
        total += scale * float((dweights[t, on] * w).sum())
        total += dloss * coef * E / (k * n * n) * float((counts[:E] * p).sum())
    return total


def backward(z, idx, counts, dweights, dloss, score=SOFTMAX, renorm=False, scale=1.0, coef=0.0):
    """dz [T, E] by the chain rule through the scores."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    k = idx.shape[1]
    n = max(int(counts[E]), 1)
    g = dloss * coef * E / (k * n * n) * counts[:E].astype(np.float64)
    dz = np.zeros((T, E))
    for t in range(T):
        on = idx[t] >= 0
        if not on.any():
            continue
        s, p = (v[0] for v in scores(z[t:t + 1], score))
        chosen, D = idx[t, on], scale * dweights[t, on]
        one_minus = 1.0 if score == SOFTMAX else np.exp(log_sigmoid(-z[t]))
        row = p * (g - (g * p).sum()) * one_minus
        if renorm:
            l = z[t, chosen] if score == SOFTMAX else log_sigmoid(z[t, chosen])
            v = np.exp(l - l.max())
            v = v / v.sum()
            part = v * (D - (D * v).sum())
            row[chosen] += part if score == SOFTMAX else part * one_minus[chosen]
        elif score == SOFTMAX:
            row[chosen] += s[chosen] * D
            row -= p * (s[chosen] * D).sum()
        else:
            row[chosen] += s[chosen] * D * one_minus[chosen]
        dz[t] = row
    return dz
