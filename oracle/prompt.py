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


ONE = 1 << 45   # the weight of the largest logit


def weights(x, T):
    """rint(2^45 exp((x - max) / T)) of one row, as Python whole numbers."""
    with np.errstate(under="ignore"):
        return [int(w) for w in np.rint(np.exp((x - x.max()) / T) * ONE)]


def sample(x, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of float64 logits: (token, its share of the kept weight), whole-number sums throughout.
    T, top_p, min_p, u: float32 values."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all() or not (0 <= T < np.inf) or u != u:
        return -1, 0.0
    if T == 0:
        return int(np.argmax(x)), 1.0
    w = weights(x, float(T))
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1:
        want = max(1, int(np.ceil(np.float64(top_p) * np.float64(sum(w[i] for i in order)))))
        kept, ahead = [], 0
        for i in order:
            if ahead >= want:
                break
            kept.append(i)
            ahead += w[i]
        order = kept
    least = int(np.ceil(min(float(min_p), 1.0) * ONE)) if min_p > 0 else 0
    order = sorted(i for i in order if w[i] >= least)
    total = sum(w[i] for i in order)
    target = min(max(int(np.floor(np.float64(u) * np.float64(total))), 0), total - 1)
    upto = 0
    for i in order:
        upto += w[i]
        if upto > target:
            return i, w[i] / total
    raise AssertionError("no token")


def unit(x, eps, scale=1.0):
    """Rows to unit length."""
    return scale * x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)


def delta_gates(b_raw, a_raw, dt_bias, a_log):
    """beta = sigmoid(b_raw), alpha = exp(-exp(a_log) softplus(a_raw + dt_bias))."""
    return 1 / (1 + np.exp(-b_raw)), discretise(a_raw, dt_bias, a_log)[1]


def delta_scan(q, k, v, beta, alpha, S):
    """The gated delta rule over one sequence, token after token; shapes as for scan()."""
    H, G = v.shape[1], q.shape[1]
    y = np.zeros(v.shape)
    S = S.copy()
    for t in range(len(v)):
        kk, qq = np.repeat(k[t], H // G, 0), np.repeat(q[t], H // G, 0)
        S = alpha[t][:, None, None] * S
        miss = v[t] - np.einsum("hpn,hn->hp", S, kk)
        S = S + (beta[t][:, None] * miss)[:, :, None] * kk[:, None, :]
        y[t] = np.einsum("hpn,hn->hp", S, qq)
    return y, S


def delta_size(q, k, v, beta, alpha, S):
    """A bound on |y| and on the rows' norms of S where |k| <= 1 and 0 <= beta <= 1: the rule's erasure, I - beta k k^T,
    lengthens no row, so a row's norm is at most |alpha| of what it was and beta |v| |k| more.  (y [n, H, P], rows [H, P])"""
    H, G = v.shape[1], q.shape[1]
    y = np.zeros(v.shape)
    z = np.sqrt((S * S).sum(-1))
    for t in range(len(v)):
        kn, qn = (np.repeat(np.sqrt((x[t] ** 2).sum(-1)), H // G)[:, None] for x in (k, q))
        z = np.abs(alpha[t])[:, None] * z + np.abs(beta[t][:, None] * v[t]) * kn
        y[t] = z * qn
    return y, z
