"""Float64 forms of the operators around the recurrence -- test
infrastructure only: the convolution and discretisation ahead of it, the scan
of a prompt.  Written from their formulas, row by row, with the magnitude of
every sum beside it, so that tests can bound rounding."""
from __future__ import annotations

import numpy as np


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def conv(x, weight, bias, hist, act=True):
    """One sequence: x [n, C], weight [C, K], hist [K - 1, C] (oldest first).
    Returns (outputs [n, C], sum of the terms' magnitudes [n, C], last K - 1
    rows [K - 1, C])."""
    n, C = x.shape
    K = weight.shape[1]
    rows = np.concatenate([hist, x])
    z = np.zeros((n, C)) if bias is None else np.tile(bias.astype(np.float64), (n, 1))
    mag = np.abs(z)
    for j in range(K):
        term = weight[:, j].astype(np.float64) * rows[j:j + n]
        z += term
        mag += np.abs(term)
    return silu(z) if act else z, mag, rows[len(rows) - (K - 1):]


def discretise(raw, dt_bias, a_log, dt_min=0.0, dt_max=np.inf):
    """dt = clamp(softplus(raw + dt_bias)), a = exp(-exp(a_log) dt); raw [n, H]."""
    x = raw.astype(np.float64) + (0.0 if dt_bias is None else dt_bias.astype(np.float64))
    dt = np.clip(np.logaddexp(x, 0.0), dt_min, dt_max)
    return dt, np.exp(-np.exp(a_log.astype(np.float64)) * dt)


def scan(q, k, v, dt, a, S):
    """One sequence, token after token: q, k [n, G, N], v [n, H, P], dt, a [n, H], S [H, P, N].
    Returns (y [n, H, P], the last state)."""
    H, G = v.shape[1], q.shape[1]
    y = np.zeros(v.shape)
    S = S.copy()
    for t in range(len(v)):
        kk, qq = np.repeat(k[t], H // G, 0), np.repeat(q[t], H // G, 0)
        S = a[t][:, None, None] * S + (dt[t][:, None] * v[t])[:, :, None] * kk[:, None, :]
        y[t] = np.einsum("hpn,hn->hp", S, qq)
    return y, S
