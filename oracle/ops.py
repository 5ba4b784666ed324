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


def logprobs_ref(logits, tokens, k, scale):
    """Per row of z = scale * logits: lse, entropy, the tokens' logprobs and the
    best k (ids, logprobs; largest first, the lower index first among equals).
    A row with a NaN or +inf: NaN and ids of -1. A row of -inf: lse and logprobs
    -inf, entropy 0. A token below 0: logprob 0; at or past the row's end: NaN."""
    T, V = logits.shape
    raw = logits.astype(np.float64)
    z = raw * scale
    bad = np.isnan(z).any(axis=1) | np.isposinf(z).any(axis=1)
    z = np.where(bad[:, None], 0.0, z)
    m = z.max(axis=1)
    empty = np.isneginf(m)
    d = np.where(empty[:, None], 0.0, z) - np.where(empty, 0.0, m)[:, None]
    e = np.exp(d)
    s = e.sum(axis=1)
    lse = np.where(empty, -np.inf, m + np.log(s))
    p = e / s[:, None]
    ent = np.where(empty, 0.0, np.log(s) - (p * np.where(p > 0, d, 0.0)).sum(axis=1))
    lp = np.where(empty[:, None], -np.inf, d - np.log(s)[:, None])
    given = np.full(T, np.nan)
    for t in range(T):
        if tokens[t] < 0:
            given[t] = 0.0
        elif tokens[t] < V:
            given[t] = lp[t, tokens[t]]
    given = np.where(bad & (tokens >= 0), np.nan, given)
    ids = np.argsort(-np.where(bad[:, None], 0.0, raw), axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(lp, ids, axis=1)
    ids = np.where(bad[:, None], -1, ids)
    nan = lambda a: np.where(bad if a.ndim == 1 else bad[:, None], np.nan, a)  # noqa: E731
    return {"lse": nan(lse), "entropy": nan(ent), "logprob": given, "top": nan(top), "ids": ids, "d": d, "p": p, "m": m}


def logprobs_grad_ref(logits, tokens, lse, entropy, g, gh, scale):
    """d sum(g logprob) + sum(gh entropy) / d logits from the formula, with the
    lse and entropy given; also p and log p."""
    z = logits.astype(np.float64) * scale
    empty = np.isneginf(lse)
    lp = z - np.where(empty, 0.0, lse)[:, None]
    p = np.where(empty[:, None], 0.0, np.exp(lp))
    live = (tokens >= 0) & (tokens < z.shape[1]) & ~empty
    gg = np.where(tokens >= 0, g, 0.0)
    hit = np.zeros_like(z)
    hit[np.arange(len(tokens))[live], tokens[live]] = 1.0
    safe = np.where(p > 0, lp, 0.0)
    d = scale * (gg[:, None] * (hit - p) - gh[:, None] * np.where(p > 0, p * (safe + entropy[:, None]), 0.0))
    return d, p, safe
