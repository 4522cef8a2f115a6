"""Rotary positions' definition (rope.h) in NumPy, with the bound that the kernels' roundings leave."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def frequencies(dims, base=10000.0, scaling="none", factor=1.0, original_tokens=1, low_turns=1.0, high_turns=32.0):
    """Angles a position, in extended precision (positions of up to 2^31 multiply them)."""
    theta = np.longdouble(base) ** (np.longdouble(-2.0) * np.arange(dims // 2, dtype=np.longdouble) / dims)
    if scaling == "linear":
        return theta / np.longdouble(factor)
    if scaling == "by_parts":
        turns = original_tokens * theta / (2 * np.longdouble("3.14159265358979323846264338327950288"))
        g = np.clip((turns - low_turns) / np.longdouble(high_turns - low_turns), 0, 1)
        return theta * (g + (1 - g) / np.longdouble(factor))
    return theta


def rotate(x, positions, theta, pairs, magnitude=1.0, back=False, eps=0.0):
    """x [b, heads, T, hd] fp64, positions [b, T]: (y, tolerance). Sines and cosines are off by up to 1.7 U (the series and
    the angle's last bit), the magnitude, its product, each product and the sum by U of (|a| + |b|) m each; `eps` is half a
    step of the storage type."""
    pi = np.longdouble("3.14159265358979323846264338327950288")
    phi = np.mod(positions.astype(np.longdouble)[..., None] * theta, 2 * pi)[:, None]
    c, s = np.cos(phi).astype(np.float64) * magnitude, np.sin(phi).astype(np.float64) * magnitude
    if back:
        s = -s
    n = 2 * len(theta)
    first, second = (slice(0, n // 2), slice(n // 2, n)) if pairs == "half" else (slice(0, n, 2), slice(1, n, 2))
    y, tol = x.copy(), np.zeros_like(x)
    a, b = x[..., first], x[..., second]
    with np.errstate(all="ignore"):
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        tol[..., first] = tol[..., second] = 6 * U * abs(magnitude) * (np.abs(a) + np.abs(b))
        tol[..., :n] += eps * np.abs(y[..., :n]) + 1e-37      # and what falls below the type's range
    return y, tol


def split(rows, heads, kvh, order):
    """(q, k, v) [b, heads, T, hd] of rows [b, T, H + 2 KVH, hd]."""
    x = rows.transpose(0, 2, 1, 3)
    if order == "contiguous":
        return x[:, :heads], x[:, heads:heads + kvh], x[:, heads + kvh:]
    b, _, t, hd = x.shape
    x = x.reshape(b, kvh, -1, t, hd)
    return x[:, :, :-2].reshape(b, heads, t, hd), x[:, :, -2], x[:, :, -1]


def join(q, k, v, order):
    """The reverse of split."""
    if order == "contiguous":
        x = np.concatenate([q, k, v], 1)
    else:
        b, kvh, t, hd = k.shape
        x = np.concatenate([q.reshape(b, kvh, -1, t, hd), k[:, :, None], v[:, :, None]], 2).reshape(b, -1, t, hd)
    return x.transpose(0, 2, 1, 3)
