"""Rotary positions with several axes: angles, tables, and the rotation of normalised heads, in float64.

Test infrastructure (see the package docstring).

A head's rotary pairs are dealt to the axes in order, dims[a] / 2 to axis a; pair i of axis a turns by
position[m, a] * theta[a]^(-2 i / dims[a]).  Pairs past the rotated columns do not turn.
"""

import numpy as np


def angles(positions, dims, thetas):
    """positions [P, axes] -> [P, sum(dims) / 2]."""
    pos = np.asarray(positions, dtype=np.float64)
    cols = []
    for a, (d, theta) in enumerate(zip(dims, thetas)):
        for i in range(d // 2):
            cols.append(pos[:, a] * np.power(float(theta), -2.0 * i / d))
    return np.stack(cols, axis=1)


def rotate(x, ang, half):
    """x [M, H, D], ang [M, R / 2]: columns 0 .. R - 1 of every head rotated, pairs (x[2i], x[2i+1]) or,
    with half, (x[i], x[i + R/2])."""
    x = np.asarray(x, dtype=np.float64)
    pairs = ang.shape[1]
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    first = np.arange(pairs) if half else 2 * np.arange(pairs)
    second = first + (pairs if half else 1)
    out = x.copy()
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., first] * s + x[..., second] * c
    return out


def norm(x, weight, eps):
    """Per-head RMSNorm; weight None: x as it is."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + float(eps)) * np.asarray(weight, dtype=np.float64)


def bound(x_normed, out, half, rot, D):
    """How far a bf16 result may be: its one rounding (half a step, 2^-8), and the fp32 work on a pair of
    normalised values -- the sum of D squares (its relative error halves under the root), the
    reciprocal root (2^-22), three products, the sine and cosine (2^-22 with the angle's rounding) and the
    rotation's products and sum -- relative to the pair's magnitudes."""
    mag = np.abs(x_normed)
    partner = mag.copy()
    n = rot // 2
    first = np.arange(n) if half else 2 * np.arange(n)
    second = first + (n if half else 1)
    partner[..., first] = partner[..., second] = mag[..., first] + mag[..., second]
    return 2.0 ** -8 * np.abs(out) + (D / 2 + 16) * 2.0 ** -24 * (1 + 2.0 ** -8) * partner + 2.0 ** -133
