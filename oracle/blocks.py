"""Block operators in 64 bits, straight from their definitions.  Inputs and
outputs are NumPy arrays, one per rank unless said otherwise.
"""

import numpy as np

E4M3_MOST = 448.0
LEAST = 2.0 ** -117


def rms_norm(s, w, eps):
    """The norm of one rank's rows s (as they are stored): (y, 1 / sqrt(mean(s^2) + eps) of each row)."""
    s, w = np.asarray(s, np.float64), np.asarray(w, np.float64)
    factor = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s * factor * w, factor


def largest(y, group=0):
    """The largest absolute value of each group of consecutive elements of a row (0: of the row), [rows, groups]."""
    group = group or y.shape[1]
    return np.stack([np.abs(y[:, i:i + group]).max(axis=1) for i in range(0, y.shape[1], group)], axis=1)


def rms_norm_grad(dy, s, w, eps, d_sum=None):
    """(d_x, d_w) of one rank's rows, term by term."""
    dy, s, w = (np.asarray(a, np.float64) for a in (dy, s, w))
    _, factor = rms_norm(s, w, eps)
    dx = np.empty_like(s)
    for t in range(s.shape[0]):
        inner = (dy[t] * w * s[t]).sum()
        dx[t] = factor[t] * dy[t] * w - s[t] * inner * factor[t] ** 3 / s.shape[1]
    if d_sum is not None:
        dx = dx + np.asarray(d_sum, np.float64)
    return dx, (dy * s * factor).sum(axis=0)
