"""Plain 64-bit restatements of the operators on rows (numpy), for the parity tests: log probabilities of
given tokens.  Shares nothing with the CUDA library.

Formulas: ember internals, softmax (a row of -inf is uniform); ember reference_forward.py main() (the greedy
token is the first of the largest logits, a NaN counting as larger than any other).
"""
from __future__ import annotations

import numpy as np


def order(row) -> np.ndarray:
    """Indices of a row in falling order of its values, NaN before all others, equal ones by their index."""
    row = np.asarray(row, np.float64)
    nan = np.isnan(row)
    return np.lexsort((np.arange(row.size), -np.where(nan, 0.0, row), ~nan))


def logprobs(logits, temperature=1.0):
    """Log probabilities [n, V] of rows of logits and the rows' entropies [n]."""
    x = np.asarray(logits, np.float64)
    t = float(np.float32(temperature))
    lp, entropy = np.full(x.shape, np.nan), np.full(x.shape[0], np.nan)
    for r in range(x.shape[0]):
        m = x[r].max()
        if np.isnan(m) or m == np.inf:
            continue
        if m == -np.inf:
            lp[r] = -np.log(x.shape[1])
        else:
            y = (x[r] - m) / t
            lp[r] = y - np.log(np.exp(y).sum())
        some = lp[r] > -np.inf
        entropy[r] = -(np.exp(lp[r][some]) * lp[r][some]).sum()
    return lp, entropy


def project(x, w, a, b, scale, ids, bias=None):
    """x [n, K] through w [N, K] with adapter ids[i] (a [A, R, K], b [A, N, R]) beside it.  Returns the outputs and,
    for error bounds, sums of magnitudes: |w| |x|, |s| |b| |a| |x| and |s| |b| summed over ranks, all [n, N]."""
    x, w, a, b = (np.asarray(t, np.float64) for t in (x, w, a, b))
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    low, ranks = np.zeros_like(y), np.zeros_like(y)
    for i, k in enumerate(np.asarray(ids)):
        if not 0 <= k < len(a):
            continue
        s = 1.0 if scale is None else float(scale[k])
        y[i] += b[k] @ (a[k] @ x[i]) * s
        low[i] = np.abs(b[k]) @ (np.abs(a[k]) @ np.abs(x[i])) * abs(s)
        ranks[i] = np.abs(b[k]).sum(-1)
    return (y if bias is None else y + np.asarray(bias, np.float64)), size, low, ranks
