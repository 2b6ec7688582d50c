"""Trees of drafted tokens against float64: outputs (replay_verify_tree), the
confirmed path (replay_accept_tree), its append (replay_append_path), and the
nodes' convolution (replay_conv_tree, replay_conv_path).

Bounds, before any run, on float32 results.  A decay over n tokens is off by n
2^-24, a dot product by N 2^-24, a sum over n entries by n 2^-24, each of the
sums of magnitudes Y.  Mamba-2: (3 n + 2 N + 64) 2^-24 Y in all, n the ring's
entries and the path's.  Gated delta rule: the weights solve a triangular
system with unit diagonal; a correction's error enters those of later entries
by beta (k_i . k_j), which for the tests' keys (random directions) is a
fraction, so eight times as much of Y, which there is the bound by row norms
(|k| = 1, beta <= 1)."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from oracle import tree as ot
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
FP4 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def _lad():
    import linear_attention_decode_amd as lad
    return lad


def _dev(a, t=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(t).to(gu.DEV)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(gu.DEV)


def random_tree(r, W):
    """Chains, bushes, several roots."""
    p = np.array([w - 1 if r.random() < 0.5 else r.integers(-1, w) if w else -1 for w in range(W)])
    p[0] = -1
    return p


class Round:
    def __init__(self, B, H, G, P, N, L, W, io, rule=0, read=None, seed=0, nodes=None, counts=None, parent=None):
        r = self.r = np.random.default_rng(seed)
        self.shape, self.W, self.L, self.rule, self.io = (B, H, G, P, N), W, L, rule, torch.bfloat16 if io == "bf16" else torch.float32
        self.layer = _lad().ReplayLayer(B, H, G, P, N, L, io_dtype=io, read_copy=read, rule="gdn" if rule else "mamba2")
        self.layer.load_checkpoint(_dev(0.5 * r.standard_normal((B, H, P, N))))
        self.parent = np.stack([random_tree(r, W) for _ in range(B)]) if parent is None else np.array(parent)
        self.n = np.array(nodes if nodes is not None else [W] * B)
        counts = r.integers(0, L + 1, B) if counts is None else np.array(counts)
        # the ring, behind a pointer that has gone round: W' = 1 appends, then rollbacks to each count
        turn = int(r.integers(0, L))
        for _ in range(turn):
            self.layer.append(1, *self.tokens(1))
        torch.cuda.synchronize()
        base = self.layer.t["base"]
        base += turn            # (as if the state had taken them: only the place in the ring matters here)
        self.layer.set_flush_skipping(False)
        ring = self.tokens(L)
        self.layer.append(L, *ring)
        self.layer.rollback(_i32(L - counts))
        self.counts = counts
        self.ring = [t.double().cpu().numpy() for t in ring]
        self.x = self.tokens(W)
        self.y = torch.full((B, W, H, P), 7.0, device=gu.DEV)

    def tokens(self, W):
        r, (B, H, G, P, N) = self.r, self.shape
        q, k, v = (r.standard_normal(s) for s in ((B, W, G, N), (B, W, G, N), (B, W, H, P)))
        dt = np.logaddexp(r.standard_normal((B, W, H)) - 1, 0)
        a = np.exp(-dt * r.uniform(0.1, 2, H))
        if self.rule:
            q, k, dt = op.unit(q, 0), op.unit(k, 0), 1 / (1 + np.exp(-r.standard_normal((B, W, H))))
        else:
            q, k = q / np.sqrt(N), k / np.sqrt(N)
        return _dev(q, self.io), _dev(k, self.io), _dev(v, self.io), _dev(dt), _dev(a)

    def state(self):
        t, (B, H, G, P, N) = self.layer.t, self.shape
        if t["s_copy"] is None:
            return t["s_master"].double().cpu().numpy()
        read = self.layer.read_copy
        if read == "bf16":
            return t["s_copy"].double().cpu().numpy()
        if read == "fp8":
            x = t["s_copy"].view(torch.float8_e4m3fn).float().double() * t["s_scale"].double()[..., None, None]
            return x.cpu().numpy()
        code = t["s_copy"].cpu().numpy()
        x = FP4[np.stack([code & 15, code >> 4], -1)].reshape(B, H, -1, 32)
        return (x * np.exp2(t["s_scale"].cpu().numpy().astype(np.float64) - 127)[..., None]).reshape(B, H, P, N)

    def run(self, y=None, n=True, stream=None):
        self.layer.verify_tree(self.W, _i32(self.parent), *self.x, self.y if y is None else y,
                               n_nodes=_i32(self.n) if n else None, stream=stream)

    def reference(self, b):
        c = self.counts[b]
        nodes = [t[b].double().cpu().numpy() for t in self.x]
        return ot.verify(self.parent[b], self.n[b], [t[b, :c] for t in self.ring], nodes, self.state()[b], self.rule)

    def check(self, seqs=None):
        torch.cuda.synchronize()
        B, H, G, P, N = self.shape
        got = self.y.double().cpu().numpy()
        for b in range(B) if seqs is None else seqs:
            y, mag = self.reference(b)
            m = self.n[b]
            n = self.counts[b] + self.W
            tol = (3 * n + 2 * N + 64) * E24 * (8 if self.rule else 1) * mag + 1e-37
            err = np.abs(got[b, :m] - y)
            assert np.all(err <= tol), (b, float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:4])
            assert np.all(got[b, m:] == 7.0)
        assert self.layer.get_error()[0] == 0


SHAPES = [(16, 16), (64, 64), (64, 128), (128, 128)]


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("L,W", [(1, 1), (5, 3), (16, 16), (16, 17), (32, 33), (8, 64), (32, 64)])
def test_trees(rule, io, P, N, L, W):
    gu.note(f"tree P={P} N={N} L={L} W={W} {io} rule {rule}")
    p = Round(4, 4, 2, P, N, L, W, io, rule, seed=L + W, nodes=[W, max(0, W - 3), 0, 1], counts=[L, 0, L // 2, max(0, L - 1)])
    before = [p.layer.t[x].clone() for x in ("pos", "base", "ring_k", "ring_v", "ring_dt", "ring_a")]
    p.run()
    p.check()
    for x, t in zip(("pos", "base", "ring_k", "ring_v", "ring_dt", "ring_a"), before):
        assert torch.equal(p.layer.t[x], t), x


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("read", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("P,N", SHAPES)
def test_trees_read_from_a_copy(rule, io, read, P, N):
    gu.note(f"tree copy {read} P={P} N={N} {io} rule {rule}")
    p = Round(3, 4, 4, P, N, 16, 21, io, rule, read, seed=P)
    p.run()
    p.check()


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("shape", ["chain", "star", "roots", "binary"])
def test_shapes_of_a_tree(rule, shape):
    gu.note(f"tree {shape} rule {rule}")
    W = 64
    parent = {"chain": np.arange(W) - 1, "star": np.minimum(np.arange(W), 1) - 1, "roots": np.full(W, -1),
              "binary": (np.arange(W) - 1) // 2}[shape]
    p = Round(2, 8, 2, 64, 128, 16, W, "bf16", rule, seed=1, parent=[parent] * 2)
    p.run(n=False)
    p.check()


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_chain_is_a_window(rule, io):
    """The window appended, verified and rolled back gives the outputs of the chain."""
    gu.note(f"tree chain against window {io} rule {rule}")
    W, L = 9, 32
    p = Round(3, 4, 2, 64, 128, L, W, io, rule, seed=8, counts=[0, 5, L - W], parent=[np.arange(W) - 1] * 3)
    p.run()
    p.check()
    y = torch.empty_like(p.y)
    p.layer.append(W, *p.x)
    p.layer.verify(W, y)
    p.layer.rollback(_i32([W] * 3))
    scale = np.stack([p.reference(b)[1] for b in range(3)])
    assert np.all(np.abs((y - p.y).double().cpu().numpy()) <= 2 * (3 * (L + W) + 2 * 128 + 64) * E24 * (8 if rule else 1) * scale)


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["q", "k", "v", "dt", "a"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_value_that_is_no_number_stays_on_its_branch(rule, io, which, value):
    """Other branches keep every bit, the node and what follows it are not finite where the rule says so; nodes past
    n_nodes reach nothing."""
    gu.note(f"tree {value} in {which} {io} rule {rule}")
    W = 24
    p = Round(2, 4, 2, 64, 128, 8, W, io, rule, seed=3, nodes=[W, 20])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    i = ["q", "k", "v", "dt", "a"].index(which)
    at = 6
    p.x[i][0, at, ..., 1] = value            # an element, or head 1
    p.x[i][1, 21] = value                    # no node
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.y[1], clean[1])
    hit = [w for w in range(W) if at in ot.path(p.parent[0], w)]
    rest = [w for w in range(W) if w not in hit]
    assert torch.equal(p.y[0, rest], clean[0, rest])
    if which == "q":
        assert not torch.isfinite(p.y[0, at]).any()                       # every head of the group has it (G = 2: element 1 of each)
        assert torch.equal(p.y[0, [w for w in hit if w != at]], clean[0, [w for w in hit if w != at]])
    elif which == "v":
        assert not torch.isfinite(p.y[0, hit][..., 1]).any()
        keep = [e for e in range(64) if e != 1]
        assert torch.equal(p.y[0, hit][..., keep], clean[0, hit][..., keep])
    elif which == "k":
        assert not torch.isfinite(p.y[0, hit]).any()
    else:
        assert not torch.isfinite(p.y[0, hit][:, 1]).any()
        assert torch.equal(p.y[0, hit][:, [0, 2, 3]], clean[0, hit][:, [0, 2, 3]])


@pytest.mark.parametrize("rule", [0, 1])
def test_decays_of_zero_and_underflow(rule):
    """a = 0 on one branch forgets what is behind it there; tiny ones underflow."""
    gu.note(f"tree zero decays rule {rule}")
    p = Round(2, 4, 2, 64, 64, 16, 40, "f32", rule, seed=4)
    a = p.x[4]
    a[0, 5] = 0.0
    a[0, 9, 2] = 0.0
    a[1, ::3] = 1e-30
    p.layer.t["ring_a"][1, 3] = 0.0
    base = p.layer.t["base"].cpu().numpy()
    if p.counts[1]:
        slots = [(int(base[1]) + j) % 16 for j in range(p.counts[1])]
        if 3 in slots:
            p.ring[4][1, slots.index(3)] = 0.0
    p.run()
    p.check()


def test_what_is_no_tree():
    gu.note("tree: bad parents and sizes")
    W = 8
    p = Round(6, 4, 2, 64, 128, 16, W, "bf16", 0, seed=2)
    p.parent[1, 3] = 3
    p.parent[2, 0] = 0
    p.parent[3, 7] = -2
    p.n[4], p.n[5] = W + 1, -1
    p.run()
    torch.cuda.synchronize()
    assert torch.isnan(p.y[1:]).all()
    word, seq = p.layer.get_error()
    lad = _lad()
    assert word == lad.SEQERR_BAD_TREE and list(seq) == [0] + [lad.SEQERR_BAD_TREE] * 5
    p.check([0])
    p.n[3] = 7                               # the bad parent is past the nodes
    p.y.fill_(7.0)
    p.run()
    torch.cuda.synchronize()
    p.layer.get_error()
    p.check([0, 3])


def test_refusals():
    """Everything a pointer, a size or a tensor can get wrong, on a live handle; nothing is launched."""
    gu.note("tree refusals")
    lad = _lad()
    p = Round(2, 4, 2, 64, 128, 16, 6, "bf16", 0)
    up, one = _i32(p.parent), _i32([1, 1])
    ok = [t.data_ptr() for t in (up, one, *p.x)]
    y = p.y.data_ptr()
    for W, status in ((0, 1), (-1, 1), (65, 2)):
        assert lad.lib.replay_verify_tree(p.layer.h, W, *ok, y, None) == status
        assert lad.lib.replay_append_path(p.layer.h, W, *ok, None) == status
    for i in (0, 2, 3, 4, 5, 6):
        for bad in (None, ok[i] + 2):
            args = list(ok)
            args[i] = bad
            assert lad.lib.replay_verify_tree(p.layer.h, 6, *args, y, None) == 1, i
            assert lad.lib.replay_append_path(p.layer.h, 6, *args, None) == 1, i
    assert lad.lib.replay_append_path(p.layer.h, 6, ok[0], None, *ok[2:], None) == 1
    assert lad.lib.replay_verify_tree(p.layer.h, 6, *ok, y + 4, None) == 1
    bad = [dict(parent=up[:, :5]), dict(parent=up.long()), dict(parent=up.cpu()), dict(y=p.y[:, :5]), dict(y=p.y.bfloat16()),
           dict(n_nodes=one[:1])]
    bad += [{n: t.transpose(0, 1)} for n, t in zip(("q", "k", "v", "dt", "a"), p.x)]
    good = dict(parent=up, y=p.y, n_nodes=one, **dict(zip(("q", "k", "v", "dt", "a"), p.x)))
    for b in bad:
        with pytest.raises(lad.ReplayError):
            p.layer.verify_tree(6, **(good | b))
    still = lad.ReplayLayer(2, 4, 2, 64, 128, 16, counters=False)
    assert lad.lib.replay_append_path(still.h, 6, *ok, None) == 1        # no arrival counters


def test_accept():
    """Paths against the oracle: many random trees over few tokens; the first of equal children; -1 is no token."""
    gu.note("accept_tree")
    r = np.random.default_rng(0)
    lad = _lad()
    for W in (1, 2, 7, 16, 63, 64):
        B = 200
        parent = np.stack([random_tree(r, W) for _ in range(B)])
        n = r.integers(0, W + 1, B)
        n[0], parent[1, 0] = W, 0
        n[2] = W + 3
        tokens, fed = r.integers(-1, 3, (B, W)), r.integers(-1, 3, (B, W))
        path, keep = _i32(np.full((B, W), 9)), _i32(np.full(B, 9))
        lad.replay_accept_tree(_i32(parent), _i32(tokens), _i32(fed), path, keep, n_nodes=_i32(n))
        path, keep = path.cpu().numpy(), keep.cpu().numpy()
        for b in range(B):
            want = ot.accept(parent[b], n[b], tokens[b], fed[b])
            assert keep[b] == len(want) and path[b].tolist() == want + [-1] * (W - len(want)), (W, b)
        none = _i32(np.full((B, W), 9))
        lad.replay_accept_tree(_i32(parent), _i32(tokens), _i32(fed), none, _i32(keep))
        assert none.cpu().numpy()[3].tolist() == (lambda w: w + [-1] * (W - len(w)))(ot.accept(parent[3], W, tokens[3], fed[3]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rule", [0, 1])
def test_append_path_is_append_of_its_tokens(io, rule):
    gu.note(f"append_path {io} rule {rule}")
    B, W, L = 5, 11, 16
    p = Round(B, 4, 2, 64, 128, L, W, io, rule, seed=6, counts=[0, 3, 16, 12, 5])
    path = [[0, 2, 5, 7], [], [4], [1, 3, 8, 10, 9], [10]]     # sequences 2 and 3 overflow
    table, keep = np.full((B, W), -1), [len(x) for x in path]
    for b, x in enumerate(path):
        table[b, :len(x)] = x
    before = {x: p.layer.t[x].clone() for x in ("pos", "base", "ring_q", "ring_k", "ring_v", "ring_dt", "ring_a")}
    p.layer.append_path(W, _i32(table), _i32(keep), *p.x)
    torch.cuda.synchronize()
    lad = _lad()
    word, seq = p.layer.get_error()
    assert word == lad.SEQERR_RING_OVERFLOW and list(seq) == [0, 0, 1, 1, 0]
    pos = before["pos"].cpu().numpy()
    want = {x: t.clone() for x, t in before.items()}
    for b in (0, 1, 4):
        for i, w in enumerate(path[b]):
            s = (pos[b] + i) % L
            want["ring_q"][b, :, s], want["ring_k"][b, :, s] = p.x[0][b, w], p.x[1][b, w]
            want["ring_v"][b, :, s] = p.x[2][b, w]
            want["ring_dt"][b, s], want["ring_a"][b, s] = p.x[3][b, w], p.x[4][b, w]
        want["pos"][b] += keep[b]
    for x, t in want.items():
        assert torch.equal(p.layer.t[x], t), x
    bad = table.copy()
    bad[0, 0], bad[1, 0], keep = W, -1, [4, 1, W + 1, -1, 0]
    p.layer.append_path(W, _i32(bad), _i32(keep), *p.x)
    torch.cuda.synchronize()
    word, seq = p.layer.get_error()
    assert word == lad.SEQERR_BAD_TREE and list(seq) == [32, 32, 32, 32, 0]
    for x, t in want.items():
        assert torch.equal(p.layer.t[x], t), x
    assert bool((p.layer.t["sync"] == 0).all())


@pytest.mark.parametrize("rule", [0, 1])
def test_flush_after_paths(rule):
    """The host's bounds on the counts: a flush behind appended paths folds what is there, whatever was kept."""
    gu.note(f"append_path then flush rule {rule}")
    B, W, L = 3, 6, 8
    lad = _lad()
    r = np.random.default_rng(5)
    p = Round(B, 4, 2, 64, 128, L, W, "f32", rule, seed=7)
    layer = lad.ReplayLayer(B, 4, 2, 64, 128, L, io_dtype="f32", rule="gdn" if rule else "mamba2")
    S = r.standard_normal((B, 4, 64, 128))
    layer.load_checkpoint(_dev(S))
    S = layer.t["s_master"].double().cpu().numpy()
    size = np.sqrt((S * S).sum(-1))
    scan = op.delta_scan if rule else op.scan
    folded = 0
    for step in range(6):
        x = p.tokens(W)
        keep = r.integers(0, 4, B)
        table = np.sort(np.stack([r.permutation(W) for _ in range(B)])[:, :4], 1)
        table = np.concatenate([table, np.full((B, W - 4), -1)], 1)
        layer.append_path(W, _i32(table), _i32(keep), *x)
        layer.flush(1)
        f = [t.double().cpu().numpy() for t in x]
        for b in range(B):
            y = [t[b, table[b, :keep[b]]] for t in f]
            S[b] = scan(*y, S[b])[1]
            for t in range(keep[b]):
                size[b] = y[4][t][:, None] * size[b] + np.abs(y[3][t][:, None] * y[2][t]) * np.repeat(
                    np.linalg.norm(y[1][t], axis=-1), 2)[:, None]
        folded += keep.sum()
        torch.cuda.synchronize()
        assert torch.equal(layer.t["base"], layer.t["pos"])
    assert folded and layer.get_error()[0] == 0
    err = np.abs(layer.t["s_master"].double().cpu().numpy() - S)
    assert np.all(err <= 8 * (3 * 24 + 2 * 128 + 64) * E24 * size[..., None])


# ---- the convolution over a tree -------------------------------------------

class Conv:
    def __init__(self, B, H, G, P, N, W, K, io, R=None, rule=0, seed=0, pad=0, lead=0, nodes=None, parent=None):
        r = np.random.default_rng(seed)
        self.io = torch.bfloat16 if io == "bf16" else torch.float32
        lad = _lad()
        C = self.C = H * P + 2 * G * N
        self.shape, self.W, self.K, self.R = (B, H, G, P, N), W, K, R or K - 1 + W
        self.cfg = lad.ReplayConfig(B, H, G, P, N, 16, lad.BF16 if io == "bf16" else lad.F32, lad.NONE, 0, rule)
        self.w, self.b = _dev(r.uniform(-.5, .5, (C, K))), _dev(r.uniform(-.5, .5, C))
        self.dt_bias, self.a_log = _dev(r.uniform(-4, -2, H)), _dev(np.log(r.uniform(1, 16, H)))
        self.conv = lad.ReplayConv(self.w, self.b, self.dt_bias, self.a_log, slots=self.R)
        rows = torch.full((B * W, lead + C + H + pad), float("nan"), dtype=self.io, device=gu.DEV)
        rows[:, lead:lead + C + H] = _dev(r.standard_normal((B * W, C + H)), self.io)
        self.x = rows[:, lead:lead + C]
        self.raw = None if rule else rows[:, lead + C:lead + C + H]
        self.state = _dev(r.standard_normal((B, self.R, C)), self.io)
        self.pos = _i32(r.integers(0, 3000, B))
        self.parent = np.stack([random_tree(r, W) for _ in range(B)]) if parent is None else np.array(parent)
        self.n = np.array(nodes if nodes is not None else [W] * B)
        self.err = _i32(np.zeros(B + 1))
        full = lambda *s, t=torch.float32: torch.full(s, 7.0, dtype=t, device=gu.DEV)  # noqa: E731
        self.q, self.k = full(B, W, G, N, t=self.io), full(B, W, G, N, t=self.io)
        self.v = full(B, W, H, P, t=self.io)
        self.dt, self.a = (None, None) if rule else (full(B, W, H), full(B, W, H))

    def run(self):
        _lad().replay_conv_tree(self.cfg, self.conv, self.W, _i32(self.parent), self.x, self.raw, self.pos, self.state, self.q,
                                self.k, self.v, self.dt, self.a, self.err, n_nodes=_i32(self.n))

    def hist(self, b):
        slots = [(int(self.pos[b]) - i) % self.R for i in range(self.K - 1, 0, -1)]
        return self.state[b].double().cpu().numpy()[slots]

    def check(self, seqs=None):
        torch.cuda.synchronize()
        B, H, G, P, N = self.shape
        e = 2.0 ** -8 if self.io == torch.bfloat16 else E24
        x = self.x.double().cpu().numpy().reshape(B, self.W, self.C)
        for b in range(B) if seqs is None else seqs:
            m = self.n[b]
            o, mag = ot.conv(self.parent[b], m, x[b], self.w.double().cpu().numpy(), self.b.double().cpu().numpy(), self.hist(b))
            got = torch.cat([t[b].reshape(self.W, -1) for t in (self.v, self.k, self.q)], 1).double().cpu().numpy()
            # K + 1 roundings of the sum, the activation's slope is below 1.1, its own function 2^-20, one rounding to the io type
            tol = 1.1 * (self.K + 1) * E24 * mag + (2.0 ** -20 + e) * np.abs(o) + 1e-37
            assert np.all(np.abs(got[:m] - o) <= tol), (b, float(np.max(np.abs(got[:m] - o) / tol)))
            assert np.all(got[m:] == 7.0)
            if self.raw is not None:
                raw = self.raw.double().cpu().numpy().reshape(B, self.W, H)[b]
                dt, a = op.discretise(raw, self.dt_bias.double().cpu().numpy(), self.a_log.double().cpu().numpy())
                gd, ga = self.dt[b].double().cpu().numpy(), self.a[b].double().cpu().numpy()
                rate = np.exp(self.a_log.double().cpu().numpy())
                slope = np.abs(raw) + np.abs(self.dt_bias.double().cpu().numpy()) + 1
                assert np.all(np.abs(gd[:m] - dt[:m]) <= (8 * E24 * dt + 2 * E24 * slope * dt)[:m])
                assert np.all(np.abs(ga[:m] - a[:m]) <= ((8 + 16 * rate * dt * (1 + slope)) * E24 * a + 1e-37)[:m])
                assert np.all(gd[m:] == 7.0) and np.all(ga[m:] == 7.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("H,G,P,N,W,pad,lead", [
    (4, 2, 64, 128, 16, 0, 0), (5, 1, 64, 64, 1, 3, 1), (3, 1, 16, 16, 64, 0, 0), (2, 2, 128, 128, 5, 1, 0),
    (6, 2, 16, 16, 33, 5, 3)])
def test_convolution(io, K, H, G, P, N, W, pad, lead):
    gu.note(f"conv_tree K={K} W={W} H={H} {io}")
    p = Conv(4, H, G, P, N, W, K, io, seed=W + K, pad=pad, lead=lead, nodes=[W, 0, max(0, W - 2), 1])
    state = p.state.clone()
    p.run()
    p.check()
    assert torch.equal(p.state, state) and p.err.cpu().eq(0).all()


def test_convolution_of_a_gated_delta_layer_and_of_many_sequences():
    gu.note("conv_tree rule 1, many sequences")
    p = Conv(300, 8, 2, 64, 128, 20, 4, "bf16", rule=1, seed=3, nodes=np.random.default_rng(1).integers(0, 21, 300))
    p.run()
    p.check(range(0, 300, 23))


def test_convolution_of_a_chain_is_the_step(io="bf16"):
    """Bit for bit: the window's convolution, and the state that its accepted rows leave."""
    gu.note("conv_tree chain")
    W, B = 7, 3
    p = Conv(B, 4, 2, 64, 128, W, 4, io, seed=9, parent=[np.arange(W) - 1] * B)
    p.run()
    q = [torch.empty_like(t) for t in (p.q, p.k, p.v, p.dt, p.a)]
    state = p.state.clone()
    _lad().replay_conv_step(p.cfg, p.conv, W, p.x, p.raw, p.pos, state, *q)
    for mine, theirs in zip((p.q, p.k, p.v, p.dt, p.a), q):
        assert torch.equal(mine, theirs)
    path = _i32(np.tile(np.arange(W), (B, 1)))
    _lad().replay_conv_path(p.cfg, p.conv, W, path, _i32([W] * B), p.x, p.pos, p.state, p.err)
    assert torch.equal(p.state, state)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R", [3, 5, 12])
def test_path_rows_into_the_state(io, R):
    gu.note(f"conv_path R={R} {io}")
    W, B = 9, 6
    p = Conv(B, 3, 1, 64, 64, W, 4, io, R=R, seed=R, pad=1)
    path = [[0, 1, 2, 3, 4, 5, 6, 7, 8], [], [3], [8, 0, 2, 4, 5, 1], [9, 1], [0, 1]]
    keep = [len(x) for x in path]
    keep[5] = W + 1
    table = np.full((B, W), -1)
    for b, x in enumerate(path):
        table[b, :len(x)] = x
    want = p.state.clone()
    x = p.x.reshape(B, W, -1)
    for b in range(4):
        for i, w in enumerate(path[b]):
            want[b, (int(p.pos[b]) + i) % R] = x[b, w]
    _lad().replay_conv_path(p.cfg, p.conv, W, _i32(table), _i32(keep), p.x, p.pos, p.state, p.err)
    torch.cuda.synchronize()
    assert torch.equal(p.state, want)
    assert p.err.cpu().tolist() == [32, 0, 0, 0, 0, 32, 32]


def test_convolution_of_what_is_no_tree():
    gu.note("conv_tree: bad trees")
    p = Conv(4, 4, 2, 64, 64, 6, 4, "f32", seed=1)
    p.parent[1, 2], p.n[2], p.parent[3, 0] = 5, 7, -3
    p.run()
    p.check([0])
    for t in (p.q, p.k, p.v, p.dt, p.a):
        assert bool((t[1:] == 7.0).all())
    assert p.err.cpu().tolist() == [32, 0, 32, 32, 32]
