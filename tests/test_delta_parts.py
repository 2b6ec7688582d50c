"""How many bits the products of replay_delta_scan's bf16 form hold, seen from its
results: the limits that tests/test_gpu_delta_parts.py sets for the kernels, and, on
a float32 emulation of the chunk algorithm with its operands cut into 8-bit parts,
that a part or a product less would break them.

The limits, before any run.  A state or an output is what some hundred float32
roundings leave, 2^-24 of a term each; they add as their root, and the largest
error over a head meets its largest value: 2^-20 of it.  y is rounded to bf16, whose
steps are 2^-8 of a value at least: a value that is off by 2^-20 of the largest rounds
otherwise than the exact one once in 2^12 for the largest and more often for the
small ones, 2^-9 in all."""
import numpy as np
import pytest

from oracle import prompt as op

STATE, FLIPS = 2.0 ** -20, 2.0 ** -9
F = np.float32
SIX = ((0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0))


def bf16(x):
    """Rounded to the nearest bf16, ties to even."""
    u = np.ascontiguousarray(x, dtype=F).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(F).reshape(np.shape(x))


def upper(x):
    return (np.ascontiguousarray(x, dtype=F).view(np.uint32) & np.uint32(0xffff0000)).view(F).reshape(np.shape(x))


def parts(x, n):
    out, x = [], np.asarray(x, F)
    for z in range(n):
        out.append(upper(x) if z + 1 < n else bf16(x))
        x = (x - out[-1]).astype(F)
    return out


def product(a, b, pairs):
    return sum(a[i].astype(np.float64) @ b[j].astype(np.float64) for i, j in pairs).astype(F)


def scan(q, k, v, beta, alpha, S, state=3, tr=SIX, y_state=3, y_tokens=SIX):
    """One head, 64 tokens at a time; q, k [n, N], v [n, P], S [P, N]: (y before its rounding, the last state).
    state: parts of S and e U in the products that make the state; tr: products of T R; y_state: parts of S in Q S^T;
    y_tokens: products of G U."""
    Y, S = np.zeros(v.shape, F), S.astype(F)
    for c in range(0, len(v), 64):
        Q, K, V, b, a = (x[c:c + 64] for x in (q, k, v, beta, alpha))
        m = len(V)
        D = np.ones((m, m), F)
        for i in range(m):
            for j in range(i - 1, -1, -1):
                D[i, j] = D[i, j + 1] * a[j + 1]
        g, e = np.cumprod(a, dtype=F), D[-1]
        A = np.tril((K.astype(np.float64) @ K.T).astype(F) * D * b[:, None], -1)
        T = (np.linalg.inv(np.eye(m) + A) * b).astype(F)
        G = np.tril((Q.astype(np.float64) @ K.T).astype(F) * D)
        R = (V - g[:, None] * sum(K.astype(np.float64) @ s for s in parts(S.T, state)).astype(F)).astype(F)
        U = product(parts(T, 3), parts(R, 3), tr)
        n = 1 + max(max(p) for p in y_tokens)
        Y[c:c + 64] = (g[:, None] * sum(Q.astype(np.float64) @ s for s in parts(S.T, 3)[:y_state])
                       + product(parts(G, n), parts(U, n), y_tokens))
        S = (g[-1] * S.T + sum(K.T.astype(np.float64) @ x for x in parts(e[:, None] * U, state))).T.astype(F)
    return Y, S


def off(y, S, want_y, want_S):
    """(the largest errors of state and y over the largest value, the share of y's that round otherwise)"""
    return (np.abs(S - want_S).max() / np.abs(want_S).max(), np.abs(y - want_y).max() / np.abs(want_y).max(),
            np.mean(bf16(y) != bf16(want_y.astype(F))))


@pytest.mark.parametrize("n,P,N", [(300, 64, 64), (300, 64, 128), (200, 128, 128)])
def test_a_part_less_is_seen(n, P, N):
    r = np.random.default_rng(n + P + N)
    q, k, v = bf16(op.unit(r.standard_normal((n, N)), 0)), bf16(op.unit(r.standard_normal((n, N)), 0)), bf16(r.standard_normal((n, P)))
    beta = (1 / (1 + np.exp(-r.standard_normal(n)))).astype(F)
    alpha = np.exp(-np.logaddexp(r.standard_normal(n) - 3, 0) * 4).astype(F)
    S = (0.5 * r.standard_normal((P, N))).astype(F)
    x = [t.astype(np.float64)[:, None] for t in (q, k, v, beta, alpha)]
    y, last = op.delta_scan(*x, S.astype(np.float64)[None])
    run = lambda **kw: off(*scan(q, k, v, beta, alpha, S, **kw), y[:, 0], last[0])  # noqa: E731
    s, o, flips = run()
    assert s < STATE and o < STATE and flips < FLIPS / 4
    three = SIX[:3]
    assert run(state=2)[0] > 2 * STATE and run(tr=three)[0] > 2 * STATE
    assert run(y_tokens=three)[2] > FLIPS
    # a state that stays as it is: y is Q S^T alone
    beta[:], alpha[:] = 0, 1
    y[:, 0], last = q.astype(np.float64) @ S.astype(np.float64).T, S[None]
    assert run()[2] < FLIPS / 4 and run(y_state=2)[2] > FLIPS
