"""Gated DeltaNet trees whose keys are finite but so long that the weights of a
path overflow float32: that reaches the nodes behind them alone, and what the
rule gives them in float32 is what they have.

Bounds, before any run.  A row of the state grows by |alpha| |1 - beta |k|^2| along
a key and takes beta |v| |k|, so with
    Z' = |alpha| (1 + beta |k|^2) Z + beta |v| |k|
every sum's terms are at most Z |q| in all; a step is off by N + 8 roundings of
them: with the system's solution, whose weights are sums of the same terms, (3 n
+ 2 N + 64) 2^-24 Z |q| for n entries, eight times as much as test_gpu_tree.py
takes.  Where Z |q| passes 2^120 float32 may overflow on the way, and does where the
value itself is past its range."""
import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests import gpu_util as gu
from tests.test_gpu_tree import E24, SHAPES, Round

pytestmark = pytest.mark.gpu

# node 0, a chain of 13 long keys behind its child 2, and nodes beside them
PARENT = [-1, 0, 0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 1, 0, 16, 15]
LONG = range(3, 16)
HIT = [*LONG, 19]
REST = [w for w in range(20) if w not in HIT]


def bound(ring, nodes, parent, w, S, heads):
    """Z |q| [H, P] of node w, from its definition above."""
    p = ot.path(parent, w)
    q, k, v, beta, alpha = [np.concatenate([r, t[p]]) for r, t in zip(ring, nodes)]
    rep = heads // k.shape[1]
    z = np.sqrt((S * S).sum(-1))
    for t in range(len(k)):
        kk = np.repeat((k[t] ** 2).sum(-1), rep)[:, None]
        b, a = beta[t][:, None], np.abs(alpha[t][:, None])
        z = a * (1 + b * kk) * z + b * np.abs(v[t]) * np.sqrt(kk)
    return z * np.repeat(np.sqrt((q[-1] ** 2).sum(-1)), rep)[:, None]


def check(p, b, nodes):
    """Node by node against float64; returns how many values were compared, and how many passed float32's range."""
    B, H, G, P, N = p.shape
    c = p.counts[b]
    ring, x, S = [t[b, :c] for t in p.ring], [t[b].double().cpu().numpy() for t in p.x], p.state()[b]
    got = p.y[b].double().cpu().numpy()
    near = past = 0
    with np.errstate(over="ignore", invalid="ignore"):
        want = ot.verify(p.parent[b], p.n[b], ring, x, S, 1)[0]
        for w in nodes:
            Z = bound(ring, x, p.parent[b], w, S, H)
            tol = 8 * (3 * (c + len(p.parent[b])) + 2 * N + 64) * E24 * Z + 1e-37
            fits, over = Z < 2.0 ** 120, np.abs(want[w]) > 2.0 ** 132
            assert np.all(np.abs(got[w] - want[w])[fits] <= tol[fits]), (b, w)
            assert not np.isfinite(got[w][over]).any(), (b, w)
            near, past = near + fits.sum(), past + over.sum()
    return near, past


def lengthen(p, b, nodes, norm, g, shared=True):
    """Keys of group g of these nodes to that length, near one direction."""
    k = p.x[1]
    N = k.shape[-1]
    d = p.r.standard_normal(N)
    for w in nodes:
        x = (d if shared else 0) + (0.2 if shared else 1) * p.r.standard_normal(N)
        k[b, w, g] = torch.from_numpy(norm * x / np.linalg.norm(x)).to(k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [30, 200, 1e10, 1e20])
@pytest.mark.parametrize("P,N", SHAPES)
def test_long_keys_stay_on_their_branch(io, norm, P, N):
    gu.note(f"tree, keys of length {norm} P={P} N={N} {io}")
    p = Round(2, 4, 2, P, N, 8, 20, io, 1, seed=int(np.log2(norm)) + N, parent=[PARENT] * 2, counts=[5, 0])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    lengthen(p, 0, LONG, norm, 1, norm < 100)
    lengthen(p, 1, LONG, norm, 0, norm < 100)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.y[:, REST], clean[:, REST])
    assert torch.equal(p.y[0, :, :2], clean[0, :, :2]) and torch.equal(p.y[1, :, 2:], clean[1, :, 2:])   # the other group
    near, past = (sum(x) for x in zip(*(check(p, b, HIT) for b in range(2))))
    assert near >= 2 * 2 * P and (norm < 1e10 or past)
    assert p.layer.get_error()[0] == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [40, 200])
def test_keys_of_some_length_without_decay(io, norm):
    """A dozen keys of this length, beta and alpha 1, are enough."""
    gu.note(f"tree, keys of length {norm} without decay {io}")
    p = Round(1, 4, 2, 64, 128, 8, 20, io, 1, seed=norm, parent=[PARENT], counts=[5])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    lengthen(p, 0, LONG, norm, 1, norm < 100)
    p.x[3][0, 3:16] = 1.0
    p.x[4][0, 3:16] = 1.0
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.y[:, REST], clean[:, REST])
    check(p, 0, HIT)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("read", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("P,N", SHAPES)
def test_long_keys_against_a_copy(io, read, P, N):
    """The same against checkpoints of fewer bits: what the rule gives comes from their values."""
    gu.note(f"tree, long keys against {read} P={P} N={N} {io}")
    p = Round(1, 4, 2, P, N, 8, 20, io, 1, read, seed=N, parent=[PARENT], counts=[3])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    # of the branch's first nodes the weights pass float32's range and the values do not
    lengthen(p, 0, LONG, 1e10, 1)
    p.x[2][0, 3:16, 2:] *= 1e-20
    p.x[4][0, 3, 2:] = 1e-30
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.y[:, REST], clean[:, REST]) and torch.equal(p.y[..., :2, :], clean[..., :2, :])
    near, past = check(p, 0, HIT)
    assert near >= 3 * 4 * P and past


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("W,nodes", [(6, 6), (64, 40)])
def test_long_keys_in_the_ring(io, P, N, W, nodes):
    """Every node is behind them: small values and states keep what the rule gives within float32's range."""
    gu.note(f"tree, long keys in the ring P={P} N={N} W={W} {io}")
    p = Round(1, 4, 2, P, N, 16, W, io, 1, seed=W, nodes=[nodes], counts=[11])
    p.layer.t["s_master"].mul_(1e-30)
    base = int(p.layer.t["base"][0])
    d = p.r.standard_normal(N)
    for j in (2, 3, 6, 7):
        slot = (base + j) % 16
        x = d + 0.2 * p.r.standard_normal(N)
        k = p.layer.t["ring_k"]
        k[0, 1, slot] = torch.from_numpy(2e7 * x / np.linalg.norm(x)).to(k)
        p.ring[1][0, j, 1] = k[0, 1, slot].double().cpu().numpy()
    for j in range(11):
        p.layer.t["ring_v"][0, :, (base + j) % 16] *= 1e-30
        p.ring[2][0, j] = p.layer.t["ring_v"][0, :, (base + j) % 16].double().cpu().numpy()
    p.run()
    torch.cuda.synchronize()
    near, _ = check(p, 0, range(nodes))
    assert near == nodes * 4 * P and bool((p.y[0, nodes:] == 7.0).all())


def test_a_captured_call_takes_either_way():
    """Replays over ordinary and over long keys, each as the eager call."""
    gu.note("tree, long keys, captured")
    p = Round(1, 4, 2, 64, 128, 8, 20, "bf16", 1, seed=3, parent=[PARENT], counts=[4])
    up = torch.tensor([PARENT], dtype=torch.int32, device=gu.DEV)
    call = lambda y: p.layer.verify_tree(20, up, *p.x, y)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(p.y)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(p.y)
    ordinary = p.x[1].clone()
    for long in (False, True, False, True):
        p.x[1].copy_(ordinary)
        if long:
            lengthen(p, 0, LONG, 1e10, 0)
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(p.y)
        call(eager)
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(eager), torch.nan_to_num(p.y))
        check(p, 0, REST)
