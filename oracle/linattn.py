"""FP64 CPU oracle of the linear attention with a decay for each head (test infrastructure only).

Per document and head h, lam = exp(slope[h]), query / key head h // (H / Hk), one token at a time:

    S_t = lam S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t
    G_t = lam G_{t+1} + scale q_t dO_t^T (+ dht at the last token),  dq_t = scale S_t dO_t,
    dk_t = G_t v_t,  dv_t = G_t^T k_t,  dh0 = lam G_first (dht of an empty document)

Parity status: pinned by tests/test_linattn_pins.py (hand-worked tokens, running sums, the pair form,
a document cut in two, central finite differences).
"""
from __future__ import annotations

import numpy as np


def _heads(x, H):
    x = np.asarray(x, dtype=np.float64)
    return np.repeat(x, H // x.shape[1], axis=1)


def linattn_fwd(q, k, v, slope, cu, h0=None, scale=1.0):
    """q, k [T, Hk, d], v [T, H, d], slope [H].  Returns (o [T, H, d], ht [N, H, d, d])."""
    v = np.asarray(v, dtype=np.float64)
    T, H, d = v.shape
    q, k, lam = _heads(q, H), _heads(k, H), np.exp(np.asarray(slope, np.float64))[:, None, None]
    N = len(cu) - 1
    o, ht = np.zeros_like(v), np.zeros((N, H, d, d))
    for n in range(N):
        S = np.zeros((H, d, d)) if h0 is None else np.array(h0[n], dtype=np.float64)
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * (q[t][:, :, None] * S).sum(1)
        ht[n] = S
    return o, ht


def linattn_bwd(q, k, v, slope, cu, dO, h0=None, dht=None, scale=1.0):
    """Gradients of sum(o dO) + sum(ht dht): dict dq, dk [T, Hk, d], dv [T, H, d], dh0 [N, H, d, d]."""
    v, dO = np.asarray(v, dtype=np.float64), np.asarray(dO, dtype=np.float64)
    T, H, d = v.shape
    Hk = np.asarray(q).shape[1]
    q, k, lam = _heads(q, H), _heads(k, H), np.exp(np.asarray(slope, np.float64))[:, None, None]
    N = len(cu) - 1
    dq, dk, dv = np.zeros_like(v), np.zeros_like(v), np.zeros_like(v)
    dh0 = np.zeros((N, H, d, d))
    for n in range(N):
        S = np.zeros((H, d, d)) if h0 is None else np.array(h0[n], dtype=np.float64)
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (S * dO[t][:, None, :]).sum(2)
        G = np.zeros((H, d, d)) if dht is None else np.array(dht[n], dtype=np.float64)
        for t in reversed(range(cu[n], cu[n + 1])):
            G = G + scale * q[t][:, :, None] * dO[t][:, None, :]
            dk[t] = (G * v[t][:, None, :]).sum(2)
            dv[t] = (G * k[t][:, :, None]).sum(1)
            G = lam * G
        dh0[n] = G
    shared = lambda x: x.reshape(T, Hk, H // Hk, d).sum(2)  # noqa: E731
    return dict(dq=shared(dq), dk=shared(dk), dv=dv, dh0=dh0)
