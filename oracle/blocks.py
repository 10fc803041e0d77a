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


# ---------------------------------------------------------------- AdamW

BLOCK = 256


def mix(x):
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x = (x * 0x9E3779B9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def chances(n, step, seed, of_means=False):
    """The chance of each of n elements at a step, in [0, 1): for the root of v, or for m."""
    key = mix(int(mix(step)) + seed)
    if of_means:
        key = key ^ np.uint64(0x6A09E667)
    pair = np.arange((n + 1) // 2, dtype=np.uint64)
    h = mix(key + pair + 0xBB67AE85 * (pair >> 32))
    return np.stack([h & 0xFFFF, h >> 16], axis=1).reshape(-1)[:n] / 65536.0


def blocks(x):
    """x in rows of BLOCK elements, zeros behind its end."""
    x = np.asarray(x, np.float64).reshape(-1)
    out = np.zeros(-(-x.size // BLOCK) * BLOCK)
    out[:x.size] = x
    return out.reshape(-1, BLOCK)


def adamw(p, g, m, v, t, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2):
    """(p, m, v) after step t, v being the mean of the squares."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    update = m / (1 - betas[0] ** t) / (np.sqrt(v / (1 - betas[1] ** t)) + eps)
    return p - lr * weight_decay * p - lr * update, m, v


def distance(x):
    """From an e4m3 value x >= 0 to the next."""
    return 2.0 ** (np.floor(np.log2(np.maximum(x, 2.0 ** -6))) - 3)


def e4m3(x):
    """x to the nearest e4m3 value (ties to even), 448 at most."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3_MOST)
    return np.sign(x) * np.minimum(np.rint(a / distance(a)) * distance(a), E4M3_MOST)


def by_chance(x, chance):
    """x >= 0 to the e4m3 value below, or where the part above and the chance reach a step to the one above."""
    x = np.minimum(x, E4M3_MOST)
    return np.minimum(np.floor(x / distance(x) + chance) * distance(x), E4M3_MOST)


def mean_codes(y, g, scale_before, beta1, chance):
    """Means in units of their new scale, y, as e4m3: to nearest, those that it would hold without a gradient by chance."""
    a = np.abs(y)
    held = (np.abs(g) < 2.0 ** -6 * scale_before) & ((1 - beta1) * a < distance(a) / 2)
    return np.where(held, np.sign(y) * by_chance(a, chance), e4m3(y)), held


def adamw8(p, g, m_code, m_scale, v_code, v_scale, t, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, seed=0):
    """One block of a parameter with 8-bit states after step t: (p, m_code, m_scale, v_code, v_scale), codes as values."""
    p, m, v = adamw(p, g, m_code * m_scale, (v_code * v_scale) ** 2, t, lr, betas, eps, weight_decay)
    r, before = np.sqrt(v), m_scale
    m_scale, v_scale = (0.0 if x < LEAST else x / E4M3_MOST for x in (np.abs(m).max(), r.max()))
    m_code, v_code = np.zeros_like(m), np.zeros_like(r)
    if m_scale:
        m_code = mean_codes(m / m_scale, g, before, betas[0], chances(m.size, t, seed, True))[0]
    if v_scale:
        v_code = np.where(r > 0, np.maximum(by_chance(r / v_scale, chances(r.size, t, seed)), 2.0 ** -9), 0.0)
    return p, m_code, m_scale, v_code, v_scale


# ---------------------------------------------------------------- experts

def moe_token(x, weights, experts, gate_up, down):
    """One token's output and, for error bounds, the sum of its terms' sizes: gate_up [E, 2I, H], down [E, H, I]."""
    y, size = np.zeros(down.shape[1]), np.zeros(down.shape[1])
    inner = down.shape[2]
    for w, e in zip(weights, experts):
        if not 0 <= e < gate_up.shape[0]:
            continue
        g, u = gate_up[e, :inner] @ x, gate_up[e, inner:] @ x
        ag, au = np.abs(gate_up[e, :inner]) @ np.abs(x), np.abs(gate_up[e, inner:]) @ np.abs(x)
        s = 1 / (1 + np.exp(-g))
        h = g * s * u
        # by how much h moves, for a relative error of one in each term of its two sums
        moved = np.abs(u) * (s + np.abs(g) * s * (1 - s)) * ag + np.abs(g * s) * au + np.abs(h) * (1 + np.abs(g))
        y += w * (down[e] @ h)
        size += np.abs(w) * (np.abs(down[e]) @ (moved + np.abs(h)))
    return y, size
