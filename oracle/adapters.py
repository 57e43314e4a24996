"""Low-rank adapters of many requests beside a shared projection, in float64.

Test infrastructure (see the package docstring).

out[m] = y[m] + sum_j weights[s, j] B[id] (A[id] x[m]) for the rows m of request s, id = ids[s, j];
id -1 adds nothing, and a row of no request keeps y.
"""

import numpy as np


def forward(x, y, a, b, offsets, ids, weights):
    """Returns (out, slack): the exact output, and the sum of the magnitudes of all products, by
    which the rounding of the intermediate sums is bounded (see ``bound``)."""
    x, y, a, b = (np.asarray(v, dtype=np.float64) for v in (x, y, a, b))
    out = y.copy()
    u_slack = np.zeros_like(y)
    k_slack = np.zeros_like(y)
    for s in range(len(offsets) - 1):
        rows = slice(offsets[s], offsets[s + 1])
        for j in range(np.shape(ids)[1]):
            i = ids[s][j]
            if i < 0:
                continue
            w = float(weights[s][j])
            u = x[rows] @ a[i].T
            out[rows] += w * (u @ b[i].T)
            u_slack[rows] += abs(w) * (np.abs(u) @ np.abs(b[i]).T)
            k_slack[rows] += abs(w) * ((np.abs(x[rows]) @ np.abs(a[i]).T) @ np.abs(b[i]).T)
    return out, u_slack, k_slack


def bound(out, u_slack, k_slack, K, ranks):
    """How far a bf16 result may be: its one rounding (half a step, 2^-8), u's split into two bf16 parts
    (2^-16) and its weighting (2^-24), and the fp32 sums -- K / 16 + 24 additions over K (tensor-core
    steps of 16 products, then up to 16 partial sums) and ranks / 8 + 2 over the ranks, each within 2^-22 of
    the running sum of magnitudes (a tensor-core step may cut off the last bits of its addends
    instead of rounding them)."""
    inner = (K / 16 + 24) * 2.0 ** -22 * k_slack + (2.0 ** -16 + 2.0 ** -24 + (ranks / 8 + 2) * 2.0 ** -22) * u_slack
    return 2.0 ** -8 * np.abs(out) + (1 + 2.0 ** -8) * inner + 2.0 ** -133
