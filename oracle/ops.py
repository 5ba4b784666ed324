"""fp64 references of the operators around the layers and the head.

Written from the operators' formulas on numpy float64 arrays; they share no
code with the kernels. ``EPS_*`` are half a step of a format relative to the
value, the largest error of one rounding.
"""

from __future__ import annotations

import numpy as np

EPS_BF16 = 2.0**-8
EPS_F32 = 2.0**-24
EPS_E4M3 = 2.0**-4
TOP_CODE = {"i8": 127.0, "e4m3": 448.0}


def rmsnorm_ref(x, r, g, eps):
    """(h, y) of y = h / sqrt(mean(h^2) + eps) * g with h = x + r. Rows are
    taken by their largest value first, so that squares stay in range; a row
    that holds an infinity or a NaN is NaN."""
    h = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
    ok = np.isfinite(h).all(axis=1, keepdims=True)
    hh = np.where(ok, h, 0.0)
    m = np.maximum(np.abs(hh).max(axis=1, keepdims=True), 1e-300)
    rms = m * np.sqrt(np.mean((hh / m) ** 2, axis=1, keepdims=True) + eps / m / m)
    y = hh / rms * (1.0 if g is None else g.astype(np.float64))
    return h, np.where(ok, y, np.nan)


def row_scale(y, fmt):
    """The scale of each row's codes: the largest magnitude over the largest code."""
    return np.abs(y).max(axis=1) / TOP_CODE[fmt]


def i8_ref(xq, x_scale, wq, w_scale):
    """(sums, C): the exact integer products (int64) and their scaled values."""
    s = (xq.astype(np.float64) @ wq.astype(np.float64).T)  # below 2^53: exact
    return s.astype(np.int64), s * x_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)
