"""FP64 CPU oracle of layer norm over the last axis (test infrastructure only).

    mean = sum v / C,  rstd = 1 / sqrt(sum (v - mean)^2 / C + eps),  xh = (v - mean) rstd
    y = xh w + b
    d = dy w:  dx = rstd (d - mean(d) - xh mean(d xh)) + dsum,  dw = sum_rows dy xh,  db = sum_rows dy

Parity status: pinned by tests/test_layernorm_pins.py (unit rows, shift and scale invariance,
central finite differences).
"""
from __future__ import annotations

import numpy as np


def _stats(v, eps):
    v = np.asarray(v, dtype=np.float64)
    mean = v.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((v - mean) ** 2).mean(-1, keepdims=True) + eps)
    return (v - mean) * rstd, mean, rstd


def layernorm_fwd(v, w=None, b=None, eps=1e-5):
    """Returns (y, mean, rstd), the statistics without the last axis."""
    xh, mean, rstd = _stats(v, eps)
    y = xh if w is None else xh * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean[..., 0], rstd[..., 0]


def layernorm_bwd(v, dy, w=None, dsum=None, eps=1e-5):
    """Returns dict dx, dw, db."""
    xh, _, rstd = _stats(v, eps)
    dy = np.asarray(dy, dtype=np.float64)
    d = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd * (d - d.mean(-1, keepdims=True) - xh * (d * xh).mean(-1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    rows = tuple(range(dy.ndim - 1))
    return dict(dx=dx, dw=(dy * xh).sum(rows), db=dy.sum(rows))
