"""Plain fp64 CPU oracle of the norms of q and k with rotary positions (test
infrastructure only), forward and gradient, for one of q and k: x [T, H, d].

Bounds on what fp32 arithmetic may differ by.  The inverse norm's sum of d
squares is a tree of at most 10 levels (10 roundings, halved by the root), then
a division by d, the addition of eps, root and reciprocal: within 8 2^-24.  A
cosine or sine is within 2^-22 of its value (2 ulp, and an angle rounded to
fp32 once, pi 2^-25), and the products and the fma of a rotated element round
three times.  In all an element's error is within C (|z_a| + |z_b|) of the
pair's magnitudes, C = 2^-20.  The gradient passes its terms through both
steps and a second sum over the head: within 4 C of the terms' magnitudes.
"""

import numpy as np

C = 2.0 ** -20


def rotate(x, r, layout, pos, inv_freq, sign=1.0, scale=1.0):
    """x [T, H, d] with its first r elements turned by sign * pos * inv_freq, times scale."""
    y = x.copy()
    if r == 0:
        return y
    ang = sign * np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = scale * np.cos(ang), scale * np.sin(ang)
    ia, ib = (np.arange(r // 2), np.arange(r // 2) + r // 2) if layout == "half" else \
        (np.arange(0, r, 2), np.arange(1, r, 2))
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def pair_size(x, r, layout, scale):
    """|z_a| + |z_b| for each element of a rotated pair, |z| elsewhere."""
    y = np.abs(x)
    if r == 0:
        return y
    ia, ib = (np.arange(r // 2), np.arange(r // 2) + r // 2) if layout == "half" else \
        (np.arange(0, r, 2), np.arange(1, r, 2))
    both = scale * (y[..., ia] + y[..., ib])
    y[..., ia] = both
    y[..., ib] = both
    return y


def inverse_norm(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    ss = (x * x).sum(-1, keepdims=True)
    return 1 / np.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)


def qk_fwd(x, norm, layout, r, pos, inv_freq, w=None, eps=1e-6, scale=1.0, rope_scale=1.0):
    """(y, bound of y); w [d]: the whole factor of norm "rms", offset included."""
    z = x * inverse_norm(x, norm, eps)
    if norm == "rms":
        z = z * w
    y = scale * rotate(z, r, layout, pos, inv_freq, 1.0, rope_scale)
    return y, C * abs(scale) * pair_size(z, r, layout, abs(rope_scale))


def qk_bwd(x, dy, norm, layout, r, pos, inv_freq, w=None, eps=1e-6, scale=1.0, rope_scale=1.0):
    """(dx, dw, bound of dx, sum of dw's terms' magnitudes); dw None unless "rms"."""
    dz = rotate(dy * scale, r, layout, pos, inv_freq, -1.0, rope_scale)
    size = pair_size(dy * scale, r, layout, abs(rope_scale))
    if norm == "none":
        return dz, None, C * size, None
    n = inverse_norm(x, norm, eps)
    dw = mag = None
    if norm == "rms":
        dw, mag = (dz * x * n).sum((0, 1)), (size * np.abs(x) * n).sum((0, 1))
        dz, size = dz * w, size * np.abs(w)
    m = x.shape[-1] if norm == "rms" else 1
    dx = n * (dz - x * (n * n / m) * (dz * x).sum(-1, keepdims=True))
    bound = 4 * C * n * (size + np.abs(x) * (n * n / m) * (size * np.abs(x)).sum(-1, keepdims=True))
    return dx, dw, bound, mag
