"""RMSNorm with the residual's addition and its gradient in numpy and 64 bits (TEST INFRASTRUCTURE)."""
import numpy as np


def forward(h, w, eps):
    """(y, rstd) of rows h [rows, cols]."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def backward(dy, h, w, rstd, dh=None):
    """(dx, dweight) for the rstd given."""
    dy, h, w, rstd = (np.asarray(v, np.float64) for v in (dy, h, w, rstd))
    hat = h * rstd[:, None]
    a = dy * w
    dx = rstd[:, None] * (a - hat * (a * hat).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * hat).sum(0)
