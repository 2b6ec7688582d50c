"""Gated DeltaNet layers ahead of the ring: their inputs (replay_delta_inputs)
and their prompts (replay_delta_scan) against float64.

Bounds, before any run: a row's squares' sum is off by N 2^-24 of itself, its
root by half that, the quotient and the product by three roundings more, then
one to the io type.  beta: two roundings and the exponential's 2^-22; alpha:
its exponent x by 8 2^-24 of itself (and what the raw sum's rounding makes of
it), the exponential's 2^-22.

The scan, in units of the bound that row norms give (|k| = 1, beta <= 1: the
erasure lengthens no row): a product of n decays is off by n 2^-24, the state
takes a sum and a product per token and one more product per chunk, a dot
product N sums: (3 n + N + 64) 2^-24; a correction's error enters later ones of
its chunk by beta (k_i . k_j), fractions for the tests' keys: eight times as
much.  With bf16 io the operands of y's products are held to 2^-15 of each
term, and y is rounded once, 2^-8 of itself."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24


def _lad():
    import linear_attention_decode_amd as lad
    return lad


def _dev(a, t=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(t).to(gu.DEV)


def _cfg(B, H, G, P, N, io, rule=1):
    lad = _lad()
    return lad.ReplayConfig(B, H, G, P, N, 16, lad.BF16 if io == "bf16" else lad.F32, lad.NONE, 0, rule)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,G,P,N,pad", [(1, 1, 1, 16, 16, 0), (7, 5, 1, 64, 64, 3), (300, 8, 4, 64, 128, 0), (33, 6, 3, 128, 128, 1),
                                           (1001, 2, 2, 16, 16, 5)])
@pytest.mark.parametrize("place", [False, True])
def test_inputs(io, T, H, G, P, N, pad, place):
    gu.note(f"delta_inputs T={T} H={H} G={G} N={N} {io}")
    r = np.random.default_rng(T)
    t = torch.bfloat16 if io == "bf16" else torch.float32
    q, k = _dev(r.standard_normal((T, G, N)), t), _dev(3 * r.standard_normal((T, G, N)), t)
    q[0] = 0.0                                             # no direction: stays zero
    raw = _dev(4 * r.standard_normal((T, 2 * H + pad)), t)
    raw[:, 2 * H:] = float("nan")
    b, a = raw[:, :H], raw[:, H:2 * H]
    bias, a_log = _dev(r.uniform(-4, 1, H)), _dev(np.log(r.uniform(1, 16, H)))
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    eps, scale = 1e-6, N ** -0.5
    want_q, want_k = op.unit(f(q), eps, scale), op.unit(f(k), eps)
    qo, ko = (q, k) if place else (torch.empty_like(q), torch.empty_like(k))
    beta, alpha = torch.empty(T, H, device=gu.DEV), torch.empty(T, H, device=gu.DEV)
    _lad().replay_delta_inputs(_cfg(1, H, G, P, N, io), T, q, k, b, a, bias, a_log, scale, eps, qo, ko, beta, alpha)
    torch.cuda.synchronize()
    e = 2.0 ** -8 if io == "bf16" else E24
    for got, want in ((qo, want_q), (ko, want_k)):
        assert np.all(np.abs(f(got) - want) <= ((N / 2 + 4) * E24 + e) * np.abs(want) * (1 + 2.0 ** -8) + 1e-37)
    wb, wa = op.delta_gates(f(b), f(a), f(bias), f(a_log))
    assert np.all(np.abs(f(beta) - wb) <= 8 * E24 * wb)
    step = np.logaddexp(f(a) + f(bias), 0)
    x = np.exp(f(a_log)) * step
    off = (8 * x + 2 * np.exp(f(a_log)) * (np.abs(f(a)) + np.abs(f(bias)))) * E24 + 4 * E24
    assert np.all(np.abs(f(alpha) - wa) <= off * wa + 1e-37)


def test_inputs_without_bias_and_with_values_that_are_no_numbers():
    """A row with a NaN is NaN, its neighbours are not; gates at their ends."""
    gu.note("delta_inputs specials")
    T, H, G, N = 4, 2, 2, 64
    q, k = torch.randn(T, G, N, device=gu.DEV), torch.randn(T, G, N, device=gu.DEV)
    q[1, 1, 5] = float("nan")
    inf = float("inf")
    b = torch.tensor([[-inf, inf], [0, -200], [200, float("nan")], [1, 2]], device=gu.DEV)
    a = torch.tensor([[-inf, inf], [0, -200], [200, float("nan")], [1, 2]], device=gu.DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    beta, alpha = torch.empty(T, H, device=gu.DEV), torch.empty(T, H, device=gu.DEV)
    _lad().replay_delta_inputs(_cfg(1, H, G, 64, N, "f32"), T, q, k, b, a, None, torch.zeros(H, device=gu.DEV), 1.0, 0.0, qo, ko,
                               beta, alpha)
    nan = torch.isnan(qo)
    assert nan[1, 1].all() and int(nan.sum()) == N and not torch.isnan(ko).any()
    assert beta.cpu()[:2].tolist() == [[0.0, 1.0], [0.5, 0.0]] and float(beta[2, 0]) == 1.0 and bool(torch.isnan(beta[2, 1]))
    assert alpha.cpu()[0].tolist() == [1.0, 0.0] and alpha.cpu()[1].tolist() == [0.5, 1.0]
    assert float(alpha[2, 0]) == 0.0 and bool(torch.isnan(alpha[2, 1]))


class Prompts:
    def __init__(self, lens, H, G, P, N, io, first=0, extra=5, resume=True, seed=0, decay=None, like=0.0, beta=None):
        r = np.random.default_rng(seed)
        lad = _lad()
        self.B, self.lens, self.io = len(lens), lens, torch.float32 if io == "f32" else torch.bfloat16
        self.shape = (H, G, P, N)
        self.T = T = max(1, first + sum(lens) + extra)
        self.cfg = _cfg(self.B, H, G, P, N, io)
        self.ends = first + np.cumsum(lens)
        self.first = first
        self.cu = torch.tensor([first, *self.ends], dtype=torch.int32, device=gu.DEV)
        k = r.standard_normal((T, G, N)) + like * r.standard_normal((1, G, N))      # like: a direction that all keys share
        self.q = _dev(op.unit(r.standard_normal((T, G, N)), 0), self.io)
        self.k = _dev(op.unit(k, 0), self.io)
        self.v = _dev(r.standard_normal((T, H, P)), self.io)
        self.beta = _dev(1 / (1 + np.exp(-r.standard_normal((T, H)))) if beta is None else beta(r, (T, H)))
        dt = np.logaddexp(r.standard_normal((T, H)) - 3, 0)
        self.alpha = _dev(np.exp(-dt * r.uniform(1, 16, H)) if decay is None else decay(r, (T, H)))
        self.s_in = _dev(0.5 * r.standard_normal((self.B, H, P, N))) if resume else None
        for t in (self.q, self.k, self.v, self.beta, self.alpha):   # rows of no sequence are read by none
            t[:first] = float("nan")
            t[self.ends[-1]:] = float("nan")
        self.err = torch.zeros(self.B + 1, dtype=torch.int32, device=gu.DEV)
        self.y = torch.full((T, H, P), 7.0, dtype=self.io, device=gu.DEV)
        self.s_out = torch.full((self.B, H, P, N), 7.0, device=gu.DEV)

    def run(self, most=None, ws="make", stream=None):
        lad = _lad()
        most = max(1, max(self.lens)) if most is None else most
        if isinstance(ws, str):   # filled with NaN: it holds nothing that a call may read before it wrote it
            n = lad.replay_delta_scan_workspace(self.cfg, self.T, most)
            ws = torch.full((n // 4,), float("nan"), device=gu.DEV) if n else None
        lad.replay_delta_scan(self.cfg, self.T, most, self.cu, self.q, self.k, self.v, self.beta, self.alpha, self.s_in,
                              self.s_out, self.y, self.err, ws, stream)
        return ws

    def rows(self, b):
        return slice(int(self.ends[b]) - self.lens[b], int(self.ends[b]))

    def reference(self, b):
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        H, G, P, N = self.shape
        S = np.zeros((H, P, N)) if self.s_in is None else f(self.s_in[b])
        x = [f(t[self.rows(b)]) for t in (self.q, self.k, self.v, self.beta, self.alpha)]
        return op.delta_scan(*x, S), op.delta_size(*x, S)

    def check(self, seqs=None):
        N = self.shape[3]
        assert self.err.cpu().eq(0).all()
        assert bool((self.y[:self.first] == 7.0).all()) and bool((self.y[int(self.ends[-1]):] == 7.0).all())
        for b in range(self.B) if seqs is None else seqs:
            n = self.lens[b]
            (y, S), (Y, Z) = self.reference(b)
            c = 8 * (3 * n + N + 64) * E24
            tol = c * Y if self.io == torch.float32 else (c + 2.0 ** -15) * Y + 2.0 ** -8 * np.abs(y)
            got, gs = self.y[self.rows(b)].double().cpu().numpy(), self.s_out[b].double().cpu().numpy()
            assert np.all(np.abs(got - y) <= tol + 1e-37), (b, float(np.max(np.abs(got - y) / (tol + 1e-37))))
            tol = c * Z[..., None] + 1e-37
            assert np.all(np.abs(gs - S) <= tol), (b, float(np.max(np.abs(gs - S) / tol)))


SHAPES = [(16, 16), (64, 64), (64, 128), (128, 128)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("lens,first,resume", [
    ([1], 0, False), ([0, 1, 2, 0], 0, True), ([15, 16, 17], 3, True), ([31, 32, 33], 0, False),
    ([63, 1, 64, 65, 0, 100], 2, True), ([200], 1, True)])
def test_ragged(io, P, N, lens, first, resume):
    gu.note(f"delta_scan {lens} P={P} N={N} {io}")
    p = Prompts(lens, 4, 2, P, N, io, first=first, resume=resume, seed=P + N + sum(lens))
    p.run()
    torch.cuda.synchronize()
    p.check()
    for b, n in enumerate(lens):     # a sequence of no tokens leaves its state
        if n == 0:
            assert torch.equal(p.s_out[b], p.s_in[b] if resume else torch.zeros_like(p.s_out[b]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H,G,P,N", [
    ([700, 1, 300], 2, 1, 64, 128), ([1111], 1, 1, 16, 16), ([513, 0, 900], 3, 3, 128, 128), ([1024, 512], 2, 2, 64, 64),
    ([2500], 4, 2, 128, 128), ([130] * 70, 3, 1, 64, 64)])
def test_long_and_many_sequences(io, lens, H, G, P, N):
    gu.note(f"delta_scan long {len(lens)} x {max(lens)} H={H} P={P} N={N} {io}")
    p = Prompts(lens, H, G, P, N, io, seed=sum(lens))
    p.run()
    torch.cuda.synchronize()
    p.check(None if len(lens) < 10 else range(0, len(lens), 9))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
def test_slow_decay_and_keys_that_are_alike(io, P, N):
    """Decays near one, keys that share a direction, strong erasure: corrections that take much of each other."""
    gu.note(f"delta_scan slow decay, like keys P={P} N={N} {io}")
    p = Prompts([400, 77], 2, 1, P, N, io, seed=4, decay=lambda r, s: np.exp(-r.uniform(0, 1e-3, s)), like=0.7,
                beta=lambda r, s: r.uniform(0.5, 1, s))
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_beta_and_alpha_at_their_ends(io):
    """beta 0 (no token), beta 1 with alpha 1 (a key's value replaced), alpha 0 (a reset), below zero and tiny ones."""
    gu.note(f"delta_scan ends {io}")

    def decay(r, s):
        pick = r.uniform(0, 1, s)
        return np.where(pick < 0.05, 0.0, np.where(pick < 0.2, 1.0, np.where(pick < 0.25, 1e-30, r.uniform(-1, 1, s))))

    def beta(r, s):
        pick = r.uniform(0, 1, s)
        return np.where(pick < 0.2, 0.0, np.where(pick < 0.5, 1.0, r.uniform(0, 1, s)))
    p = Prompts([150, 97, 64], 4, 2, 64, 128, io, seed=5, decay=decay, beta=beta)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("which", ["q", "k", "v", "beta", "alpha"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_no_numbers(io, P, N, which, value):
    """They reach no earlier token, no other sequence, head or column, and what they have to reach is not finite."""
    gu.note(f"delta_scan {value} in {which} P={P} N={N} {io}")
    lens = [90, 40]
    p = Prompts(lens, 4, 2, P, N, io, seed=6)
    p.run()
    torch.cuda.synchronize()
    y, S = p.y.clone(), p.s_out.clone()
    t = getattr(p, which)
    at = 45
    if which in ("q", "k"):
        t[at, 1, 3] = value              # heads 2 and 3
        heads, cols = [2, 3], slice(None)
    elif which == "v":
        t[at, 2, 3] = value
        t[at + 3, 2, 5] = value          # a second one, a little later
        heads, cols = [2], [3]
    else:
        t[at, 2] = value
        heads, cols = [2], slice(None)
    p.run()
    torch.cuda.synchronize()
    others = [h for h in range(4) if h not in heads]
    assert torch.equal(p.y[:, others], y[:, others]) and torch.equal(p.s_out[:, others], S[:, others])
    assert torch.equal(p.y[90:], y[90:]) and torch.equal(p.s_out[1], S[1])
    e = 2.0 ** -7 if io == "bf16" else 2.0 ** -14      # chunks that begin elsewhere: other sums
    near = lambda a, b: bool(((a.float() - b.float()).abs() <= e * (b.float().abs() + 1)).all())  # noqa: E731
    assert near(p.y[:at], y[:at])
    if which == "q":
        assert not torch.isfinite(p.y[at, heads]).any()
        assert near(p.y[at + 1:90], y[at + 1:90]) and near(p.s_out, S)
        return
    assert not torch.isfinite(p.y[at:90, heads][..., cols]).any()
    assert not torch.isfinite(p.s_out[0, heads][:, cols]).any()
    if which == "v":
        rest = [c for c in range(P) if c not in (3, 5)]
        assert near(p.y[:90, 2][:, rest], y[:90, 2][:, rest]) and near(p.s_out[0, 2, rest], S[0, 2, rest])
        assert near(p.y[:at + 3, 2, 5], y[:at + 3, 2, 5]) and not torch.isfinite(p.y[at + 3:90, 2, 5]).any()


def test_bad_ranges_leave_their_sequences():
    gu.note("delta_scan bad ranges")
    lad = _lad()
    for cu, most, bad in (([0, 40, 35, 95], 64, [1]), ([-1, 40, 60, 95], 64, [0]), ([0, 40, 60, 500], 64, [2]),
                          ([0, 70, 90, 95], 64, [0])):
        p = Prompts([40, 20, 35], 4, 2, 64, 64, "bf16", extra=0)
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        p.run(most=most)
        torch.cuda.synchronize()
        want = [lad.SEQERR_BAD_RANGE if b in bad else 0 for b in range(3)]
        assert p.err.cpu().tolist() == [lad.SEQERR_BAD_RANGE] + want, cu
        for b in bad:
            assert bool((p.s_out[b] == 7.0).all())


def test_graph_replays_and_other_streams():
    """A captured call serves other prompts and lengths (up to the capture's longest); eager work between the replays."""
    gu.note("delta_scan graph")
    p = Prompts([300, 20, 64], 4, 2, 64, 128, "bf16", seed=1, extra=40)
    ws = p.run(most=384)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        p.run(most=384, ws=ws)
    side.synchronize()
    with torch.cuda.graph(g):
        p.run(most=384, ws=ws)
    for i, lens in enumerate(([384, 0, 1], [1, 130, 200], [64, 64, 64])):
        q = Prompts(lens, 4, 2, 64, 128, "bf16", seed=20 + i, extra=p.T - sum(lens))
        for n in ("q", "k", "v", "beta", "alpha", "s_in", "cu"):
            getattr(p, n).copy_(getattr(q, n))
        p.lens, p.ends = lens, q.ends
        p.y.fill_(7.0)
        p.s_out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        p.check()
        (p.v.float() * 2).sum().item()


def test_scan_refusals_of_the_binding():
    lad = _lad()
    p = Prompts([40, 20], 4, 2, 64, 64, "bf16")
    good = dict(cu_seqlens=p.cu, q=p.q, k=p.k, v=p.v, beta=p.beta, alpha=p.alpha, s_in=p.s_in, s_out=p.s_out, y=p.y, err=p.err)
    for bad in (dict(q=p.q[:-1]), dict(k=p.k.float()), dict(v=p.v.transpose(0, 1)), dict(beta=p.beta[:, :2]), dict(alpha=None),
                dict(s_in=p.s_in.cpu()), dict(s_out=p.s_in), dict(y=p.y.float()), dict(err=p.err[1:]), dict(cu_seqlens=p.cu.long())):
        with pytest.raises(lad.ReplayError):
            lad.replay_delta_scan(p.cfg, p.T, 64, **(good | bad))
    with pytest.raises(lad.ReplayError):
        lad.replay_delta_scan(_cfg(2, 4, 2, 64, 64, "bf16", rule=0), p.T, 64, **good)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_in_pieces_and_on_through_the_ring(io):
    """A prompt in two pieces is the prompt; from its state the ring's steps go on as the rule does."""
    gu.note(f"delta_scan pieces, then steps {io}")
    lad = _lad()
    n, cut, steps = 150, 83, 12
    p = Prompts([n + steps], 4, 2, 64, 128, io, resume=False, seed=11, extra=0)
    whole, size = p.reference(0)
    layer = lad.ReplayLayer(1, 4, 2, 64, 128, 8, io_dtype=io, rule="gdn")
    S = None
    for lo, hi in ((0, cut), (cut, n)):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device=gu.DEV)
        out = torch.empty(1, 4, 64, 128, device=gu.DEV)
        need = lad.replay_delta_scan_workspace(layer.cfg, hi - lo, hi - lo)
        ws = torch.empty(need, dtype=torch.uint8, device=gu.DEV) if need else None
        layer.scan(hi - lo, hi - lo, cu, *(t[lo:hi].contiguous() for t in (p.q, p.k, p.v, p.beta, p.alpha)), S, out, p.y[lo:hi], ws)
        S = out
    layer.load_checkpoint(S)
    y = torch.empty(steps, 4, 64, device=gu.DEV)
    for t in range(steps):
        layer.step(*(x[n + t:n + t + 1].contiguous() for x in (p.q, p.k, p.v, p.beta, p.alpha)), y[t:t + 1])
    torch.cuda.synchronize()
    assert layer.get_error()[0] == 0
    c = 8 * (3 * (n + steps) + 128 + 64) * E24
    Y, want = size[0], whole[0]
    tol = c * Y[:n] + (0 if io == "f32" else 2.0 ** -15 * Y[:n] + 2.0 ** -8 * np.abs(want[:n]))
    assert np.all(np.abs(p.y[:n].double().cpu().numpy() - want[:n]) <= tol)
    assert np.all(np.abs(y.double().cpu().numpy() - want[n:]) <= c * Y[n:])
