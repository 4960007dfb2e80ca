"""MXFP4 and the products with it, in numpy and 64 bits (TEST INFRASTRUCTURE).

Written from the format's definition: E2M1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4,
6, one scale 2^e per 32 columns.  Scales are step-major, [ceil(cols/256), rows, 8].
"""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
CEIL, FLOOR = 0, 1


def scale_exp(amax, rule=CEIL):
    """The exponent for a group's largest magnitude (finite float64)."""
    if amax == 0.0:
        return -127
    mant, ex = np.frexp(amax)  # amax = mant * 2^ex, 1/2 <= mant < 1
    e = int(ex) - 3            # floor(log2 amax) - 2
    if rule == CEIL and amax > np.ldexp(6.0, e):
        e += 1
    return max(e, -127)


def encode(v):
    """E2M1 code of float64 values: nearest magnitude, ties to the code with an even last bit, clipped at 6."""
    a = np.abs(v)[..., None]
    d = np.abs(a - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (pick | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def quant(x, rule=CEIL):
    """x [rows, cols] (cols padded with zeros to 32) -> (q [rows, cols/2], s [ceil(cols/256), rows, 8])."""
    x = np.asarray(x, np.float64)
    rows = x.shape[0]
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % 32)))
    groups = x.reshape(rows, -1, 32)
    bad = ~np.isfinite(groups).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, groups)).max(-1)
    e = np.vectorize(lambda a: scale_exp(a, rule), otypes=[np.int64])(amax) if amax.size else amax.astype(np.int64)
    with np.errstate(invalid="ignore"):
        codes = encode(np.where(bad[..., None], 0.0, groups) * np.exp2(-e.astype(np.float64))[..., None])
    codes = codes.reshape(rows, -1, 2)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    s = np.pad(s, ((0, 0), (0, -s.shape[1] % 8))).reshape(rows, -1, 8).transpose(1, 0, 2)
    return codes[..., 0] | (codes[..., 1] << 4), np.ascontiguousarray(s)


def row_scales(s, groups):
    """The scale bytes as [rows, groups]."""
    return s.transpose(1, 0, 2).reshape(s.shape[1], -1)[:, :groups]


def dequant(q, s):
    """The values, float64 [rows, cols]; NaN where the scale byte is 255."""
    rows = q.shape[0]
    code = np.stack([q & 15, q >> 4], 2).reshape(rows, -1)
    v = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
    b = row_scales(s, code.shape[1] // 32).astype(np.float64)
    return v * np.repeat(np.where(b == 255, np.nan, np.exp2(b - 127)), 32, axis=1)


def gemm(av, bv):
    """av [M, K] times bv [N, K] transposed, float64, and the sum of the products' magnitudes."""
    return av @ bv.T, np.abs(av) @ np.abs(bv).T
