"""Plain 64-bit restatement of the paged-cache operators (numpy; attend_all: torch), for the parity
tests: which keys a query sees, attention over a sequence's pages, and the
append step (per-head RMS norm, rotate-half RoPE).  Shares nothing with the
CUDA library.

Formulas: ember reference_forward.py forward() (grouped-query heads, causal
softmax) and rope(); PII-Tracer serving/reference_forward.py forward() (q / k
norm before RoPE); ember internals, softmax.
"""
from __future__ import annotations

import numpy as np
import torch


def visible(pos: int, n_keys: int, window: int = 0, sinks: int = 0) -> np.ndarray:
    """Bool [n_keys]: the keys that a query at position `pos` sees."""
    key = np.arange(n_keys)
    ok = key <= pos
    if window > 0:
        ok &= (key > pos - window) | (key < sinks)
    return ok


def gather(pages: np.ndarray, table_row: np.ndarray, rows: np.ndarray) -> np.ndarray:
    """Rows `rows` of one sequence from pages [n_pages, NKV, P, D] -> [len(rows), NKV, D]."""
    P = pages.shape[2]
    return pages[table_row[rows // P], :, rows % P].astype(np.float64)


def attend(q, k_pages, v_pages, table_row, length, pos, window=0, sinks=0, scale=None):
    """Attention of the query rows q [n, NH, D] at positions pos [n] over the first
    `length` keys of one sequence.  Returns out, lse, and for error bounds the
    absolute means sum_j p_j |v_j| [n, NH, D] and the largest sum |q k| scale."""
    q = np.asarray(q, np.float64)
    n, NH, D = q.shape
    NKV = k_pages.shape[1]
    G = NH // NKV
    scale = D ** -0.5 if scale is None else float(np.float32(scale))
    out = np.zeros_like(q)
    mean = np.zeros_like(q)
    lse = np.full((n, NH), -np.inf)
    big = 0.0
    for i in range(n):
        rows = np.nonzero(visible(int(pos[i]), length, window, sinks))[0]
        if rows.size == 0:
            continue
        k, v = gather(k_pages, table_row, rows), gather(v_pages, table_row, rows)
        for h in range(NH):
            kk, vv = k[:, h // G], v[:, h // G]
            s = (kk @ q[i, h]) * scale
            live = s > -np.inf                       # a score of -inf has no weight
            if not live.any():
                continue
            big = max(big, float((np.abs(kk[live]) @ np.abs(q[i, h])).max() * abs(scale)))
            m = s[live].max()
            p = np.exp(s[live] - m)
            total = p.sum()
            lse[i, h] = m + np.log(total)
            out[i, h] = p @ vv[live] / total
            mean[i, h] = p @ np.abs(vv[live]) / total
    return out, lse, mean, big


def attend_all(q, k, v, pos, window=0, sinks=0, scale=None):
    """The same for many rows at once, on torch f64 tensors of any device and with the
    sequence's keys gathered: q [n, NH, D], k, v [length, NKV, D], pos [n].  Returns out,
    lse, sum_j p_j |v_j| and, per row and head, the largest sum |q k| |scale| over the
    keys that count."""
    n, NH, D = q.shape
    G = NH // k.shape[1]
    scale = D ** -0.5 if scale is None else float(np.float32(scale))
    key = torch.arange(k.shape[0], device=q.device)[None]
    at = pos[:, None]
    hidden = key > at
    if window > 0:
        hidden |= (key <= at - window) & (key >= sinks)
    out, mean = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, NH), -torch.inf, dtype=q.dtype, device=q.device)
    big = torch.zeros_like(lse)
    for h in range(NH):
        kk, vv = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kk.T * scale).masked_fill(hidden, -torch.inf)
        live = s > -torch.inf                        # hidden, or without weight
        m = s.amax(-1, keepdim=True).clamp(min=-1e300) if k.shape[0] else s.new_zeros(n, 1)
        p = torch.where(live, (s - m).exp(), 0.0)
        total = p.sum(-1, keepdim=True)
        some = total > 0
        p = p / torch.where(some, total, 1.0)
        used = live.any(0)                           # what no row sees may hold anything
        vv = torch.where(used[:, None], vv, 0.0)
        out[:, h], mean[:, h] = p @ vv, p @ vv.abs()
        lse[:, h] = torch.where(some, m + torch.where(some, total, 1.0).log(), -torch.inf)[:, 0]
        if k.shape[0]:
            size = q[:, h].abs() @ torch.where(used[:, None], kk, 0.0).abs().T * abs(scale)
            big[:, h] = torch.where(live, size, 0.0).amax(-1)
    return out, lse, mean, big


def norm_rope(x, w, eps, cos, sin, dtype=np.float64):
    """x [n, heads, D]: RMS norm per head (w None: none), then rotate-half by
    cos / sin [n, D/2].  With dtype float32 every product and sum is rounded
    separately, as the f32 kernels do without a norm."""
    x = np.asarray(x, dtype)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + dtype(eps)) * np.asarray(w, dtype)
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    c, s = np.asarray(cos, dtype)[:, None], np.asarray(sin, dtype)[:, None]
    return np.concatenate((a * c - b * s, b * c + a * s), -1)
