"""FP64 CPU oracle of the norm and rotation of queries and keys (test infrastructure only).

Per token t and head vector x of D channels:
    norm:  n = x w / sqrt(mean(x^2) + eps)      (else n = x)
    pair i < R / 2 (halves: channels i, R / 2 + i; neighbours: 2 i, 2 i + 1) with a = pos[t] freq[i]:
    (y1, y2) = scale (n1 cos a - n2 sin a, n1 sin a + n2 cos a);  other channels y = n

Parity status: pinned by tests/test_rope_pins.py (lengths and relative positions, a quarter turn by
hand, both layouts a permutation apart, central finite differences).
"""
from __future__ import annotations

import numpy as np


def _pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, R // 2 + i)


def _turn(n, pos, freq, interleaved, scale, back):
    R = 2 * len(freq)
    a, b = _pairs(R, interleaved)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = scale * np.cos(ang), scale * np.sin(ang) * (-1.0 if back else 1.0)
    y = n.copy()
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., a] * s + n[..., b] * c
    return y


def rope_fwd(x, pos, freq, w=None, norm=False, eps=1e-6, interleaved=False, scale=1.0):
    """x [T, heads, D] -> the same shape."""
    n = np.array(x, dtype=np.float64)
    if norm:
        n = n / np.sqrt((n ** 2).mean(-1, keepdims=True) + eps)
        if w is not None:
            n = n * np.asarray(w, np.float64)
    return _turn(n, pos, freq, interleaved, scale, False)


def rope_bwd(x, pos, freq, dy, w=None, norm=False, eps=1e-6, interleaved=False, scale=1.0):
    """Returns (dx, dw); dw is None without the norm."""
    d = _turn(np.array(dy, dtype=np.float64), pos, freq, interleaved, scale, True)
    if not norm:
        return d, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    xh = x * r
    dw = (d * xh).sum((0, 1))
    g = d if w is None else d * np.asarray(w, np.float64)
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), dw
