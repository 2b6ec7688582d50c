"""Float64 forms of the tree calls -- test infrastructure only: a tree of
drafted tokens behind a ring, node by node from its path."""
from __future__ import annotations

import numpy as np

from oracle import prompt as op


def path(parent, w):
    """The nodes from a root down to w."""
    out = []
    while w >= 0:
        out.append(w)
        w = int(parent[w])
    return out[::-1]


def is_tree(parent, n, W):
    return 0 <= n <= W and all(-1 <= parent[w] < w for w in range(n))


def verify(parent, n, ring, nodes, S, rule):
    """One sequence.  ring, nodes: (q, k, v, dt, a), tokens first (the ring's q is not used); S [H, P, N].  Returns y
    [n, H, P] and a bound on its magnitude, each node by the recurrence over the ring and its path."""
    scan, size = (op.delta_scan, op.delta_size) if rule else (op.scan, None)
    y, mag = [], []
    for w in range(n):
        p = path(parent, w)
        x = [np.concatenate([r, t[p]]) for r, t in zip(ring, nodes)]
        y.append(scan(*x, S)[0][-1])
        mag.append(size(*x, S)[0][-1] if rule else op.scan(*map(np.abs, x), np.abs(S))[0][-1])
    shape = (0, *nodes[2].shape[1:])
    return (np.stack(y), np.stack(mag)) if n else (np.zeros(shape), np.zeros(shape))


def conv(parent, n, x, weight, bias, hist, act=True):
    """One sequence: each node's convolution over its path behind hist [K - 1, C].  (outputs [n, C], magnitudes)"""
    out, mag = [], []
    for w in range(n):
        o, m, _ = op.conv(x[path(parent, w)], weight, bias, hist, act)
        out.append(o[-1])
        mag.append(m[-1])
    return (np.stack(out), np.stack(mag)) if n else (np.zeros((0, x.shape[1])),) * 2


def accept(parent, n, tokens, fed):
    """The confirmed path, from node 0."""
    if not is_tree(parent, n, len(parent)) or n == 0:
        return []
    out = [0]
    while True:
        t = tokens[out[-1]]
        child = [w for w in range(n) if parent[w] == out[-1] and fed[w] == t and t >= 0]
        if not child:
            return out
        out.append(child[0])
