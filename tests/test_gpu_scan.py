"""The recurrence over packed prompts (replay_scan) against float64.

Bounds, before any run, in units of the sums of magnitudes: Y, the outputs,
and Z, the states, of the recurrence on |q|, |k|, |v|, |a| (every partial sum
lies below them).  A decay over n tokens is a product of n factors, off by
n 2^-24; the state takes a product and a sum per token and one more product
per chunk, a dot product N sums, a weight four products.  So a float32 result
is off by at most (3 n + N + 64) 2^-24 of Y or Z.  With bf16 io the state and
the weights of earlier tokens enter their products as bf16, 2^-8 of Y at
most, and y is rounded to bf16, 2^-8 of itself; states keep the float32
bound (their products take v, scaled, in parts that hold 24 bits)."""
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


def _cfg(B, H, G, P, N, io):
    lad = _lad()
    return lad.ReplayConfig(B, H, G, P, N, 16, lad.BF16 if io == "bf16" else lad.F32, lad.NONE, 0)


def _workspace(cfg, T, most):
    """The workspace, filled with NaN: it holds nothing that a call may read before it wrote it."""
    n = _lad().replay_scan_workspace(cfg, T, most)
    return torch.full((n // 4,), float("nan"), device=gu.DEV) if n else None


class Prompts:
    def __init__(self, lens, H, G, P, N, io, first=0, extra=5, resume=True, seed=0, decay=None):
        r = np.random.default_rng(seed)
        self.B, self.lens, self.io = len(lens), lens, torch.bfloat16 if io == "bf16" else torch.float32
        self.shape = (H, G, P, N)
        self.T = T = max(1, first + sum(lens) + extra)
        self.cfg = _cfg(self.B, H, G, P, N, io)
        self.ends = first + np.cumsum(lens)
        self.cu = torch.tensor([first, *self.ends], dtype=torch.int32, device=gu.DEV)
        dev = lambda a, t=None: torch.from_numpy(a.astype(np.float32)).to(t or torch.float32).to(gu.DEV)  # noqa: E731
        act = lambda x: x / (1 + np.exp(-x))  # noqa: E731
        self.q, self.k = (dev(act(r.standard_normal((T, G, N))), self.io) for _ in range(2))
        self.v = dev(act(r.standard_normal((T, H, P))), self.io)
        dt = np.logaddexp(r.standard_normal((T, H)) - 3, 0)
        self.dt = dev(dt)
        self.a = dev(np.exp(-dt * r.uniform(1, 16, H)) if decay is None else decay(r, (T, H)))
        self.s_in = dev(0.5 * r.standard_normal((self.B, H, P, N))) if resume else None
        for t in (self.q, self.k, self.v, self.dt, self.a):   # rows of no sequence are read by none
            t[:first] = float("nan")
            t[self.ends[-1]:] = float("nan")
        self.first = first
        self.err = torch.zeros(self.B + 1, dtype=torch.int32, device=gu.DEV)
        self.y = torch.full((T, H, P), 7.0, dtype=self.io, device=gu.DEV)
        self.s_out = torch.full((self.B, H, P, N), 7.0, device=gu.DEV)

    def run(self, most=None, ws="make", stream=None):
        most = max(1, max(self.lens)) if most is None else most
        ws = _workspace(self.cfg, self.T, most) if isinstance(ws, str) else ws
        _lad().replay_scan(self.cfg, self.T, most, self.cu, self.q, self.k, self.v, self.dt, self.a, self.s_in, self.s_out,
                           self.y, self.err, ws, stream)
        return ws

    def reference(self, b, mag=False):
        rows = slice(int(self.ends[b]) - self.lens[b], int(self.ends[b]))
        f = (lambda t: np.abs(t.double().cpu().numpy())) if mag else (lambda t: t.double().cpu().numpy())
        H, G, P, N = self.shape
        S = np.zeros((H, P, N)) if self.s_in is None else f(self.s_in[b])
        return op.scan(*(f(t[rows]) for t in (self.q, self.k, self.v, self.dt, self.a)), S)

    def check(self, seqs=None):
        N = self.shape[3]
        assert self.err.cpu().eq(0).all()
        assert bool((self.y[:self.first] == 7.0).all()) and bool((self.y[int(self.ends[-1]):] == 7.0).all())
        for b in range(self.B) if seqs is None else seqs:
            n = self.lens[b]
            rows = slice(int(self.ends[b]) - n, int(self.ends[b]))
            (y, S), (Y, Z) = self.reference(b), self.reference(b, True)
            c = (3 * n + N + 64) * E24
            tol = c * Y if self.io == torch.float32 else (c + 2.0 ** -8) * Y + 2.0 ** -8 * np.abs(y)
            got, gs = self.y[rows].double().cpu().numpy(), self.s_out[b].double().cpu().numpy()
            assert np.all(np.abs(got - y) <= tol + 1e-37), (b, float(np.max(np.abs(got - y) / (tol + 1e-37))))
            assert np.all(np.abs(gs - S) <= c * Z + 1e-37), (b, float(np.max(np.abs(gs - S) / (c * Z + 1e-37))))


SHAPES = [(16, 16), (64, 64), (64, 128), (128, 128)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("lens,first,resume", [
    ([1], 0, False), ([0, 1, 2, 0], 0, True), ([15, 16, 17], 3, True), ([31, 32, 33], 0, False),
    ([63, 1, 64, 65, 0, 100], 2, True), ([200], 1, True)])
def test_ragged(io, P, N, lens, first, resume):
    gu.note(f"scan {lens} P={P} N={N} {io}")
    p = Prompts(lens, 4, 2, P, N, io, first=first, resume=resume, seed=P + N + sum(lens))
    p.run()
    torch.cuda.synchronize()
    p.check()
    for b, n in enumerate(lens):     # a sequence of no tokens leaves its state
        if n == 0:
            assert torch.equal(p.s_out[b], p.s_in[b] if resume else torch.zeros_like(p.s_out[b]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H,G,P,N", [
    ([700, 1, 300], 2, 1, 64, 128), ([1111], 1, 1, 16, 16), ([513, 0, 900], 3, 3, 128, 128), ([1024, 512], 2, 2, 64, 64)])
def test_long_sequences_in_segments(io, lens, H, G, P, N):
    gu.note(f"scan segments {lens} H={H} P={P} N={N} {io}")
    p = Prompts(lens, H, G, P, N, io, seed=sum(lens))
    assert p.run() is not None       # the workspace form
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slow_decay(io):
    """Decays near one: what the first tokens left is still whole at the end of every segment."""
    gu.note(f"scan slow decay {io}")
    p = Prompts([800, 77], 2, 1, 64, 128, io, seed=4, decay=lambda r, s: np.exp(-r.uniform(0, 1e-3, s)))
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays_of_zero_below_zero_and_underflow(io):
    """a = 0 forgets all before it, exactly; negative, above one and tiny ones follow the recurrence."""
    gu.note(f"scan odd decays {io}")

    def decay(r, s):
        x = r.uniform(-1, 1.01, s)
        pick = r.uniform(0, 1, s)
        x[pick < 0.1] = 0.0
        x[pick > 0.9] = 1e-30
        return x

    p = Prompts([130, 40], 4, 2, 64, 64, io, seed=8, decay=decay)
    p.run()
    torch.cuda.synchronize()
    p.check()
    # a reset at the last token: the state is that token's own product
    p.a[int(p.ends[0]) - 1] = 0.0
    p.run()
    torch.cuda.synchronize()
    t = int(p.ends[0]) - 1
    u = (p.v[t].float() * p.dt[t].unsqueeze(-1)).double()
    want = u.unsqueeze(-1) * p.k[t].double().repeat_interleave(2, 0).unsqueeze(1)
    assert bool(((p.s_out[0].double() - want).abs() <= 4 * E24 * want.abs()).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
def test_whole_numbers_are_exact(io, P, N):
    """Whole numbers small enough that every sum is exact, resets and steps among them: states to the bit, and y."""
    gu.note(f"scan whole numbers P={P} N={N} {io}")
    p = Prompts([97, 64, 3], 4, 2, P, N, io, seed=2)
    r = np.random.default_rng(7)
    dev = lambda a, t: torch.from_numpy(a.astype(np.float32)).to(t).to(gu.DEV)  # noqa: E731
    T, (H, G) = p.T, p.shape[:2]
    few = lambda s: (r.integers(-1, 2, s) * (r.uniform(0, 1, s) < 0.2))  # noqa: E731
    p.q, p.k, p.v = dev(few((T, G, N)), p.io), dev(few((T, G, N)), p.io), dev(few((T, H, P)), p.io)
    p.dt = dev(2.0 ** r.integers(0, 2, (T, H)), torch.float32)
    p.a = dev(r.choice([1.0, 1.0, -1.0, 0.0], (T, H), p=[0.5, 0.3, 0.17, 0.03]), torch.float32)
    p.s_in = dev(r.integers(-3, 4, p.s_in.shape), torch.float32)
    p.run()
    torch.cuda.synchronize()
    for b in range(p.B):
        y, S = p.reference(b)
        assert np.array_equal(p.s_out[b].double().cpu().numpy(), S), b
        rows = slice(int(p.ends[b]) - p.lens[b], int(p.ends[b]))
        # whole numbers below 256: as bf16 they are themselves, whatever order they were summed in
        assert np.abs(S).max() < 256 and np.abs(y).max() < 2 ** 24
        want = torch.from_numpy(y).to(p.io)
        assert torch.equal(p.y[rows].cpu(), want), b


def test_ranges():
    """Ranges that decrease, leave 0..T or are longer than max_len: flagged, their rows and states left as they were."""
    lad = _lad()
    gu.note("scan bad ranges")
    for cu, most, bad in (([0, 10, 5, 20], 20, [1]), ([0, 10, 20, 50], 40, [2]), ([-1, 8, 8, 20], 20, [0]),
                          ([0, 10, 30, 40], 15, [1]), ([0, 50, 3, 20], 50, [0, 1])):
        p = Prompts([10, 10, 15], 2, 1, 16, 16, "bf16", seed=1)
        assert p.T == 40
        p.cu = torch.tensor(cu, dtype=torch.int32, device=gu.DEV)
        for t in (p.q, p.k, p.v, p.dt, p.a):
            t[35:] = 0.5
        p.run(most=most)
        torch.cuda.synchronize()
        err = p.err.cpu().tolist()
        assert err[0] == lad.SEQERR_BAD_RANGE and [b for b in range(3) if err[1 + b]] == bad, cu
        assert all(bool((p.s_out[b] == 7.0).all()) for b in bad)
        taken = torch.zeros(40, dtype=torch.bool)
        for b in range(3):
            if b not in bad:
                taken[cu[b]:cu[b + 1]] = True
                assert bool(p.s_out[b].isfinite().all()) and not bool((p.s_out[b] == 7.0).all())
        assert bool((p.y[~taken.to(gu.DEV)] == 7.0).all()), cu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_nan_stays_in_its_sequence_and_head(io, value):
    """What is not finite reaches the outputs from its own token on, in its head and column only."""
    gu.note(f"scan {value} {io}")
    p = Prompts([50, 40], 2, 2, 64, 64, io, seed=3)
    p.v[20, 0, 5] = value
    p.run()
    torch.cuda.synchronize()
    y, S = p.y, p.s_out
    assert not y[20:50, 0, 5].isfinite().any() and not S[0, 0, 5].isfinite().all()
    assert y[20, 0, 5].isnan() if value != value else True
    y2 = y.clone()
    y2[20:50, 0, 5] = 0.0
    assert y2[:90].isfinite().all() and S[1].isfinite().all() and S[0, 1].isfinite().all()
    clean = Prompts([50, 40], 2, 2, 64, 64, io, seed=3)
    clean.run()
    torch.cuda.synchronize()
    y2[20:50, 0, 5] = clean.y[20:50, 0, 5]
    assert torch.equal(y2[:90], clean.y[:90]) and torch.equal(S[0, 1], clean.s_out[0, 1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_in_pieces(io):
    """A prompt in pieces that hand their states on is the prompt at once, within the bound of one of them each."""
    gu.note(f"scan in pieces {io}")
    p = Prompts([300], 4, 2, 64, 128, io, seed=6)
    p.run()
    whole = p.y.clone(), p.s_out.clone()
    lad, S = _lad(), p.s_in
    y = torch.full_like(p.y, 7.0)
    for lo, hi in ((0, 1), (1, 34), (34, 290), (290, 300)):
        nxt = torch.empty_like(p.s_out)
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device=gu.DEV)
        lad.replay_scan(p.cfg, hi - lo, hi - lo, cu, p.q[lo:hi], p.k[lo:hi], p.v[lo:hi], p.dt[lo:hi], p.a[lo:hi], S, nxt,
                        y[lo:hi], p.err, _workspace(p.cfg, hi - lo, hi - lo))
        S = nxt
    torch.cuda.synchronize()
    p.y, p.s_out = y, S
    p.check()
    p.y, p.s_out = whole
    p.check()


def test_replays_and_streams():
    """A captured scan (segments, workspace) replayed on new inputs equals the eager call, bit for bit, on its own
    stream; two calls at once on two streams, a workspace each, do too."""
    gu.note("scan in a graph")
    p = Prompts([700, 40], 2, 1, 64, 128, "bf16", seed=12)
    ws = _workspace(p.cfg, p.T, 700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p.run(ws=ws)
    for i in range(3):
        fresh = Prompts([700, 40], 2, 1, 64, 128, "bf16", seed=20 + i)
        for n in ("q", "k", "v", "dt", "a", "s_in"):
            getattr(p, n).copy_(getattr(fresh, n))
        fresh.run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.s_out, fresh.s_out) and torch.equal(p.y[:740], fresh.y[:740]), i
    two = [Prompts([700, 40], 2, 1, 64, 128, "bf16", seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in two]
    torch.cuda.synchronize()
    spaces = [_workspace(t.cfg, t.T, 700) for t in two]
    torch.cuda.synchronize()
    for t, s, w in zip(two, streams, spaces):
        t.run(ws=w, stream=s)
    torch.cuda.synchronize()
    for i, t in enumerate(two):
        alone = Prompts([700, 40], 2, 1, 64, 128, "bf16", seed=20 + i)
        alone.run()
        torch.cuda.synchronize()
        assert torch.equal(t.s_out, alone.s_out) and torch.equal(t.y[:740], alone.y[:740])


def test_refusals():
    lad = _lad()
    gu.note("scan refusals")
    p = Prompts([700], 1, 1, 16, 16, "bf16")
    need = lad.replay_scan_workspace(p.cfg, p.T, 700)
    assert need > 0
    for ws in (None, torch.empty(need - 4, dtype=torch.uint8, device=gu.DEV)):
        with pytest.raises(lad.ReplayError, match="status 1"):
            p.run(ws=ws)
    with pytest.raises(lad.ReplayError):
        p.run(ws=torch.empty(need, dtype=torch.uint8))
    p.s_out = p.s_in                                  # in place
    with pytest.raises(lad.ReplayError, match="status 1"):
        p.run()
    p.s_out = torch.empty_like(p.s_in)
    p.y = p.y.float()
    with pytest.raises(lad.ReplayError):
        p.run()


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("H,G", [(3, 1), (3, 3), (5, 1)])
@pytest.mark.parametrize("lens", [[63, 1, 64, 65, 0, 100], [700, 3]])
def test_odd_heads_per_group(lens, H, G, N):
    """64-wide heads in bf16 go two to a workgroup; groups of an odd number of heads, one."""
    gu.note(f"scan odd heads {lens} H={H} G={G} N={N}")
    p = Prompts(lens, H, G, 64, N, "bf16", first=2, seed=H + N + sum(lens))
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("H,G,P,N", [(3, 1, 64, 64), (3, 3, 64, 128), (2, 1, 128, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_stays_in_its_column(value, H, G, P, N):
    gu.note(f"scan {value} H={H} G={G} P={P} N={N}")
    p, clean = (Prompts([90, 20], H, G, P, N, "bf16", seed=5) for _ in range(2))
    p.v[37, H - 1, 40] = value
    p.run()
    clean.run()
    torch.cuda.synchronize()
    assert not p.y[37:90, H - 1, 40].isfinite().any() and not p.s_out[0, H - 1, 40].isfinite().all()
    p.y[37:90, H - 1, 40] = clean.y[37:90, H - 1, 40]
    p.s_out[0, H - 1, 40] = clean.s_out[0, H - 1, 40]
    assert torch.equal(p.y[:110], clean.y[:110]) and torch.equal(p.s_out, clean.s_out)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B", [63, 64, 65, 130])
def test_many_sequences(io, B):
    """Around the number of sequences that are put in order of their lengths; equal lengths, and none, among them."""
    gu.note(f"scan of {B} sequences {io}")
    lens = [(7 * b * b) % 41 for b in range(B)]
    p = Prompts(lens, 2, 1, 64, 64, io, seed=B)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("io,lens,H,G,P,N", [
    ("bf16", [384], 2, 1, 64, 64), ("bf16", [383, 2], 2, 1, 64, 64), ("f32", [192, 191], 1, 1, 64, 64),
    ("f32", [193], 1, 1, 16, 16), ("bf16", [2049, 64, 65, 0], 8, 1, 64, 64), ("bf16", [1537], 1, 1, 128, 128),
    ("f32", [1300, 1299], 2, 2, 16, 16)])
def test_segments_of_a_chunk(io, lens, H, G, P, N):
    """Around the lengths from which few heads are split, into segments as short as a chunk; more than eight of them."""
    gu.note(f"scan short segments {lens} H={H} P={P} N={N} {io}")
    p = Prompts(lens, H, G, P, N, io, seed=sum(lens) + H)
    ws = p.run()
    torch.cuda.synchronize()
    assert (ws is None) == (max(lens) == 383)
    p.check()


@pytest.mark.parametrize("H,G,P,N", [(4, 2, 64, 64), (4, 2, 64, 128), (3, 1, 64, 128), (2, 1, 128, 128)])
@pytest.mark.parametrize("lens", [[150, 33, 1], [1100]])
def test_sums_of_either_sign(lens, H, G, P, N):
    """bf16 io, terms that cancel (q, k, v of either sign, slow decay): y is a float32 sum rounded once.

    The state and the weights enter y's products as two bf16 parts each, the first cut, the second rounded: what they
    leave out of x is at most 2^-7 |x| of a cut to 8 bits, and of that the 2^-8 of a rounding; 2^-15 of Y with the float32
    sums' (3 n + N + 64) 2^-24, then the rounding of y itself."""
    gu.note(f"scan of either sign {lens} H={H} G={G} P={P} N={N}")
    p = Prompts(lens, H, G, P, N, "bf16", seed=sum(lens) + N + H, decay=lambda r, s: np.exp(-r.uniform(0, 0.02, s)))
    r = np.random.default_rng(1)
    for t in (p.q, p.k, p.v):
        t.copy_(torch.from_numpy(r.standard_normal(tuple(t.shape)).astype(np.float32)).to(p.io))
    p.run()
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        rows = slice(int(p.ends[b]) - n, int(p.ends[b]))
        (y, _), (Y, _) = p.reference(b), p.reference(b, True)
        e = ((3 * n + N + 64) * E24 + 2.0 ** -15) * Y
        off = np.abs(p.y[rows].double().cpu().numpy() - y) / (e + 2.0 ** -8 * (np.abs(y) + e) + 1e-37)
        assert np.all(off <= 1), (b, float(off.max()), float((off > 1).mean()))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
def test_growth_and_decay_in_turns(io, P, N):
    """Decays far above and below one, whose products over consecutive tokens stay finite (2^96 at most) while those of
    stretches that lie apart would not; every second chunk starts with a reset."""
    gu.note(f"scan growth and decay P={P} N={N} {io}")
    p = Prompts([128, 60], 4, 2, P, N, io, seed=P + N, decay=lambda r, s: r.uniform(0.5, 1.0, s))
    for s0 in (0, 64, 128):
        p.a[s0 + 16:s0 + 32], p.a[s0 + 32:s0 + 48], p.a[s0 + 48:s0 + 60] = 64.0, 1 / 64, 64.0
        p.a[s0 + 60:s0 + 64] = 0.75
    p.a[64] = 0.0
    p.a[188:] = float("nan")
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("start", [0.0, 1e-10])
def test_growth_then_a_reset(io, start):
    """A product of 1e28 over a prompt in segments, from no state and from a small one; then a reset, and growth again."""
    gu.note(f"scan growth then reset from {start} {io}")
    p = Prompts([700, 90], 2, 1, 64, 128, io, seed=14, decay=lambda r, s: np.full(s, 1.1))
    p.s_in.mul_(start)
    p.v[:500] = 0.0
    p.a[650] = 0.0
    assert p.run() is not None
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("lens,H,G,P,N", [([255, 64, 65, 0], 3, 1, 64, 128), ([224, 223], 2, 2, 128, 128), ([193, 192], 5, 1, 64, 64)])
def test_four_segments_of_a_short_prompt(lens, H, G, P, N):
    """float32, between three chunks and four: a segment a chunk, the last of any length."""
    gu.note(f"scan four segments {lens} H={H} P={P} N={N}")
    p = Prompts(lens, H, G, P, N, "f32", seed=sum(lens))
    ws = p.run()
    torch.cuda.synchronize()
    assert ws.numel() == 3 * p.B * H * (P * N + 1)
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N,H,G,lens", [(64, 128, 4, 2, [90, 20]), (16, 16, 2, 1, [70, 9]), (128, 128, 2, 2, [130]), (64, 64, 3, 1, [500, 70])])
@pytest.mark.parametrize("name", ["q", "k", "v", "dt", "a", "s_in"])
def test_what_is_not_finite_reaches_what_the_recurrence_lets_it(io, P, N, H, G, lens, name):
    """Outputs and states are finite where the float64 recurrence's are, and nowhere else."""
    gu.note(f"scan not finite {name} P={P} N={N} H={H} {io}")
    for value in (float("inf"), -float("inf"), float("nan")):
        p = Prompts(lens, H, G, P, N, io, seed=N + H)
        for b, at in enumerate((37, 2)[:len(lens)]):
            t = int(p.ends[b]) - lens[b] + at
            if name in "qk":
                getattr(p, name)[t, b % G, 3] = value
            elif name == "v":
                p.v[t, H - 1 - b, 9] = value
            elif name == "s_in":
                p.s_in[b, b, 2, 7] = value
            else:
                getattr(p, name)[t, H - 1 - b] = value
        p.run()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            with np.errstate(invalid="ignore"):
                y, S = p.reference(b)
            rows = slice(int(p.ends[b]) - n, int(p.ends[b]))
            assert np.array_equal(p.y[rows].isfinite().cpu().numpy(), np.isfinite(y)), (value, b)
            assert np.array_equal(p.s_out[b].isfinite().cpu().numpy(), np.isfinite(S)), (value, b)
