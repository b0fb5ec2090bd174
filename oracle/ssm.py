"""FP64 CPU oracle of the selective state-space scan (test infrastructure only: the same import
rules as the rest of this package apply).

Per document of the pack, channel c (of group g = c // (C / G)) and state s:

    delta = softplus(dt + dt_bias)   (softplus False: delta = dt + dt_bias)
    h_t[c, s] = exp(delta A[c, s]) h_{t-1}[c, s] + delta u[t, c] B[t, g, s],   h before the document: h0
    y0[t, c] = sum_s Cm[t, g, s] h_t[c, s] + D[c] u[t, c],   y = y0 silu(z)   (no z: y = y0)

The recurrence is evaluated token by token.  The backward of L = sum(y dy) + sum(ht dht) walks it
backwards: with dY = dy silu(z) and G_t = dL/dh_t,

    G_t = Cm_t dY_t + exp(delta_{t+1} A) G_{t+1}   (dht at the document's last token)

and every gradient is the product rule applied to the three lines above.

Parity status: pinned by tests/test_ssm_pins.py -- a constant decay against the geometric sum, a
document's prefix sum at zero decay, the pack against its documents alone, a document cut in two
with the state handed over, and central finite differences of every gradient.
"""
from __future__ import annotations

import numpy as np


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _prep(u, dt, A, B, Cm, D, dt_bias, z, softplus):
    u, dt, A, B, Cm, D, dt_bias, z = (_f(x) for x in (u, dt, A, B, Cm, D, dt_bias, z))
    T, C = u.shape
    S = A.shape[1]
    B, Cm = B.reshape(T, -1, S), Cm.reshape(T, -1, S)
    group = np.arange(C) // (C // B.shape[1])
    raw = dt if dt_bias is None else dt + dt_bias
    delta = np.logaddexp(raw, 0.0) if softplus else raw
    return u, A, B, Cm, (np.zeros(C) if D is None else D), z, raw, delta, group


def ssm_fwd(u, dt, A, B, Cm, cu_seqlens, *, D=None, dt_bias=None, z=None, h0=None, softplus=True):
    """Returns (y [T, C], ht [N, C, S])."""
    y, ht, _, _ = _forward(u, dt, A, B, Cm, cu_seqlens, D, dt_bias, z, h0, softplus)
    return y, ht


def _forward(u, dt, A, B, Cm, cu_seqlens, D, dt_bias, z, h0, softplus):
    u, A, B, Cm, D, z, _, delta, group = _prep(u, dt, A, B, Cm, D, dt_bias, z, softplus)
    cu = np.asarray(cu_seqlens, dtype=np.int64)
    N, (T, C), S = len(cu) - 1, u.shape, A.shape[1]
    y0, hs, ht = np.zeros((T, C)), np.zeros((T, C, S)), np.zeros((N, C, S))
    for n in range(N):
        h = np.zeros((C, S)) if h0 is None else np.array(_f(h0)[n])
        for t in range(cu[n], cu[n + 1]):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * u[t])[:, None] * B[t][group]
            hs[t] = h
            y0[t] = (Cm[t][group] * h).sum(1) + D * u[t]
        ht[n] = h
    y = y0 if z is None else y0 * z * _sigmoid(z)
    return y, ht, y0, hs


def ssm_bwd(u, dt, A, B, Cm, cu_seqlens, dy, *, D=None, dt_bias=None, z=None, h0=None, dht=None,
            softplus=True):
    """Returns dict du, ddt, dA, dB, dC, dD, ddt_bias, dh0 and (with z) dz."""
    _, _, y0, hs = _forward(u, dt, A, B, Cm, cu_seqlens, D, dt_bias, z, h0, softplus)
    shape = np.asarray(B).shape
    u, A, B, Cm, D, z, raw, delta, group = _prep(u, dt, A, B, Cm, D, dt_bias, z, softplus)
    cu = np.asarray(cu_seqlens, dtype=np.int64)
    N, (T, C), S, G = len(cu) - 1, u.shape, A.shape[1], B.shape[1]
    dY, out = _f(dy), {}
    if z is not None:
        s = _sigmoid(z)
        out["dz"] = dY * y0 * (s + z * s * (1.0 - s))
        dY = dY * z * s
    du, ddelta, dA = D * dY, np.zeros((T, C)), np.zeros((C, S))
    dB, dC, dh0 = np.zeros((T, G, S)), np.zeros((T, G, S)), np.zeros((N, C, S))
    for n in range(N):
        g = np.zeros((C, S)) if dht is None else np.array(_f(dht)[n])
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            prev = hs[t - 1] if t > cu[n] else (np.zeros((C, S)) if h0 is None else _f(h0)[n])
            g = g + Cm[t][group] * dY[t][:, None]
            np.add.at(dC[t], group, dY[t][:, None] * hs[t])
            np.add.at(dB[t], group, g * (delta[t] * u[t])[:, None])
            gB = (g * B[t][group]).sum(1)
            a = np.exp(delta[t][:, None] * A)
            du[t] += delta[t] * gB
            ddelta[t] = u[t] * gB + (g * prev * a * A).sum(1)
            dA += g * prev * a * delta[t][:, None]
            g = g * a
        dh0[n] = g
    ddt = ddelta * _sigmoid(raw) if softplus else ddelta
    out.update(du=du, ddt=ddt, dA=dA, dB=dB.reshape(shape), dC=dC.reshape(shape),
               dD=(dY * u).sum(0), ddt_bias=ddt.sum(0), dh0=dh0)
    return out
