"""The float64 forms of oracle/prompt.py against other forms of the same
definitions: the scan against the eager oracle of the decode path, the
convolution against numpy's, sampling against its definition by cumulated
probabilities on rows without ties or borders."""
import numpy as np

from oracle import prompt as op
from oracle import runs


def test_scan_is_the_eager_recurrence():
    r = np.random.default_rng(0)
    T, H, G, P, N = 9, 4, 2, 16, 16
    x = {"q": r.standard_normal((T, 1, G, N)), "k": r.standard_normal((T, 1, G, N)), "v": r.standard_normal((T, 1, H, P)),
         "dt": r.uniform(0, 1, (T, 1, H)), "a": r.uniform(0, 1, (T, 1, H))}
    want = runs.standard(x, np.zeros((1, H, P, N)))[:, 0]
    y, S = op.scan(*(x[n][:, 0] for n in ("q", "k", "v", "dt", "a")), np.zeros((H, P, N)))
    assert np.allclose(y, want, rtol=1e-12, atol=1e-12)
    assert np.allclose(np.einsum("hpn,hn->hp", S, np.repeat(x["q"][-1, 0], 2, 0)), want[-1])


def test_convolution():
    r = np.random.default_rng(1)
    x, w, b, hist = r.standard_normal((12, 5)), r.standard_normal((5, 4)), r.standard_normal(5), r.standard_normal((3, 5))
    z, mag, last = op.conv(x, w, b, hist, act=False)
    rows = np.concatenate([hist, x])
    for c in range(5):
        assert np.allclose(z[:, c], np.convolve(rows[:, c], w[c, ::-1], "valid") + b[c])
    assert np.all(mag >= np.abs(z)) and np.array_equal(last, x[-3:])
    assert np.array_equal(op.conv(x[:1], w, b, hist)[2], np.concatenate([hist[1:], x[:1]]))
    assert np.allclose(op.conv(x, w, b, hist)[0], z / (1 + np.exp(-z)))


def test_discretise():
    raw = np.array([[-800.0, 0.0, 900.0]])
    dt, a = op.discretise(raw, None, np.zeros(3))
    assert np.allclose(dt, [[0.0, np.log(2), 900.0]]) and np.allclose(a, np.exp(-dt))
    assert np.allclose(op.discretise(raw, np.ones(3), np.zeros(3), 0.5, 10)[0], [[0.5, np.log1p(np.e), 10]])


def test_sampling():
    r = np.random.default_rng(2)
    x = r.standard_normal(50) * 2
    p = np.exp(x - x.max())
    p /= p.sum()
    for u in r.uniform(0, 1, 50).astype(np.float32):
        tok, share = op.sample(x, u)
        assert tok == np.searchsorted(np.cumsum(p), u, side="right") and abs(share - p[tok]) < 1e-12
    by = np.argsort(-x)
    assert {op.sample(x, u, top_k=3)[0] for u in np.linspace(0, 1, 400, dtype=np.float32)} == set(by[:3])
    n = int(np.searchsorted(np.cumsum(p[by]), 0.8)) + 1
    assert {op.sample(x, u, top_p=0.8)[0] for u in np.linspace(0, 1, 4000, dtype=np.float32)} == set(by[:n])
    assert {op.sample(x, u, min_p=0.3)[0] for u in np.linspace(0, 1, 400, dtype=np.float32)} == set(np.flatnonzero(p >= 0.3 * p.max()))
    assert op.sample(x, 0.9, T=0) == (by[0], 1.0) and op.sample(np.zeros(9), 0.999, top_k=2)[0] == 1
    assert op.sample(x * np.nan, 0.5)[0] == -1 and op.sample(x - np.inf, 0.5)[0] == -1
