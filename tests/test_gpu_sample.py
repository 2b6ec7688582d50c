"""replay_sample against whole-number arithmetic on the host: tokens equal,
shares to float32 rounding (their quotient is taken in float64 from sums that
differ by a unit in 2^45 per token at most: 2^-24 of itself, and 2^-20 for
the last weights' own rounding, rint of a value of few units)."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
F = np.float32


def _lad():
    import linear_attention_decode_amd as lad
    return lad


def _dev(a, t):
    return torch.from_numpy(np.array(a)).to(t).to(gu.DEV)


class Rows:
    """B sequences of W positions of V logits; rows `pad` elements apart beyond V, `shift` elements off alignment."""

    def __init__(self, x, io, W=1, pad=0, shift=0):
        n, V = x.shape
        self.B, self.W, self.V = n // W, W, V
        t = torch.bfloat16 if io == "bf16" else torch.float32
        buf = torch.full((shift + n * (V + pad),), float("nan"), dtype=t, device=gu.DEV)
        self.logits = buf[shift:].view(self.B, W, V + pad)[:, :, :V]
        self.logits.copy_(_dev(x.reshape(self.B, W, V).astype(F), torch.float32).to(t))
        self.x = self.logits.double().cpu().numpy().reshape(n, V)

    def run(self, u, T=None, k=None, p=None, mp=None, fed=None, stream=None):
        B, W = self.B, self.W
        f = lambda a: None if a is None else _dev(np.broadcast_to(np.asarray(a, F), (B,)), torch.float32)  # noqa: E731
        self.u = np.broadcast_to(np.asarray(u, F).reshape(-1, W) if np.ndim(u) else F(u), (B, W))
        self.set = [np.broadcast_to(np.asarray(d if a is None else a, t), (B,)) for a, d, t in
                    ((T, 1, F), (k, 0, np.int32), (p, 1, F), (mp, 0, F))]
        self.tokens = torch.full((B, W), -7, dtype=torch.int32, device=gu.DEV)
        self.probs = torch.full((B, W), -7.0, device=gu.DEV)
        self.rej = None if fed is None else torch.full((B,), -7, dtype=torch.int32, device=gu.DEV)
        kk = None if k is None else _dev(np.broadcast_to(np.asarray(k, np.int32), (B,)), torch.int32)
        need = _lad().replay_sample_workspace(B, W, self.V)
        ws = torch.full((need,), 0x5a, dtype=torch.uint8, device=gu.DEV) if need else None
        _lad().replay_sample(self.logits, _dev(self.u, torch.float32), self.tokens, f(T), kk, f(p), f(mp), self.probs,
                             None if fed is None else _dev(fed.astype(np.int32), torch.int32), self.rej, ws, stream)
        torch.cuda.synchronize()
        return self

    def check(self, what=""):
        tok, pr = self.tokens.cpu().numpy(), self.probs.cpu().numpy()
        for r in range(self.B * self.W):
            b, w = divmod(r, self.W)
            T, k, p, mp = (s[b] for s in self.set)
            want, share = op.sample(self.x[r], self.u[b, w], T, int(k), p, mp)
            case = (what, r, "T %g k %d p %g min %g u %.9g V %d" % (T, k, p, mp, self.u[b, w], self.V))
            assert tok[b, w] == want, (case, int(tok[b, w]), want)
            assert abs(pr[b, w] - share) <= 2.0 ** -20 * share + 1e-13, (case, float(pr[b, w]), share)


def _logits(r, n, V, spread=2.5):
    return r.standard_normal((n, V)) * spread - 1.05 * np.log(r.permutation(V) + 2.7)


# T, k, p, min_p
SETTINGS = [(1, 0, 1, 0), (0.7, 50, 1, 0), (0.8, 0, 0.9, 0), (1.2, 0, 1, 0.05), (0.9, 40, 0.95, 0.02), (1, 1, 1, 0), (1, 0, 0, 0),
            (1, 0, -1, 0), (1.5, 7, 0.5, 0.3), (1, 0, 0.999, 0), (3, 1000, 0.7, 0), (1, 0, 1, 1), (1, 0, 1, 2), (0, 5, 0.5, 0.1),
            (1e-6, 0, 0.9, 0), (1e30, 0, 0.5, 0), (1, -3, 1.5, -1)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 9, 64, 300, 511, 513, 1000, 4099])
def test_settings(io, V):
    r = np.random.default_rng(V)
    gu.note(f"sample settings V={V} {io}")
    rows = Rows(_logits(r, len(SETTINGS), V), io)
    for u in (0.0, 0.37, 1 - 2.0 ** -24):
        rows.run(u, *(np.array([s[i] for s in SETTINGS]) for i in range(4))).check()
    rows.run(r.uniform(0, 1, len(SETTINGS))).check("no settings")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (0, 1), (3, 5), (1, 0)])
def test_rows_off_alignment(io, pad, shift):
    r = np.random.default_rng(3)
    gu.note(f"sample pad={pad} shift={shift} {io}")
    for V in (5, 1001):
        rows = Rows(_logits(r, 6, V), io, W=2, pad=pad, shift=shift)
        rows.run(r.uniform(0, 1, 6), k=[0, 20, 3], p=[0.9, 1, 0.8]).check()


@pytest.mark.parametrize("io,V", [("bf16", 131072), ("f32", 50021), ("bf16", 262144), ("f32", 262143)])
def test_large(io, V):
    r = np.random.default_rng(V)
    gu.note(f"sample V={V} {io}")
    T, k, p, mp = [1, 0.8, 1.1, 1, 0.7, 1], [0, 50, 0, 6000, 1000, 0], [1, 0.9, 0.95, 0.9, 1, 0.9999], [0, 0, 0, 0, 0.01, 0]
    Rows(_logits(r, 6, V), io).run(r.uniform(0, 1, 6), T, k, p, mp).check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ties(io):
    """Equal logits in the thousands: the lowest indexes stay, whichever path finds the end of the prefix."""
    r = np.random.default_rng(5)
    gu.note(f"sample ties {io}")
    V = 20011
    x = np.zeros((8, V))
    x[1] = r.integers(0, 2, V)
    x[2] = r.integers(0, 3, V) * 0.5
    x[3, :9000] = 1.0
    x[4] = np.where(r.uniform(0, 1, V) < 0.5, -0.0, 0.0)
    x[5] = r.integers(0, 40, V) / 8
    x[6, 17] = 30.0
    x[7] = -np.inf
    x[7, r.integers(0, V, 5000)] = 2.0
    rows = Rows(x, io)
    for T, k, p in ((1, 5, 1), (1, 5000, 1), (1, 12345, 0.5), (1, 0, 0.5), (0.5, 0, 0.01), (1, 0, 1), (1, 9000, 0.9), (0, 0, 1)):
        rows.run(r.uniform(0, 1, 8), T, k, p).check((T, k, p))
    rows.run(r.uniform(0, 1, 8), mp=0.7).check("min_p")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_masks_and_rows_without_an_answer(io):
    gu.note(f"sample masks {io}")
    V, r = 700, np.random.default_rng(1)
    low = float(torch.finfo(torch.bfloat16 if io == "bf16" else torch.float32).min)
    x = _logits(r, 9, V)
    x[0, 100:] = -np.inf
    x[1] = -np.inf
    x[2, 5] = np.nan
    x[3, 699] = np.inf
    x[4] = -np.inf
    x[4, 333] = -4.0
    x[5] = low
    x[6, :650] = low
    x[7] = np.where(r.uniform(0, 1, V) < 0.99, -np.inf, x[7])
    x[8, 3] = -np.nan
    rows = Rows(x, io)
    for T, k, p in ((1, 0, 1), (0.7, 30, 0.9), (1, 0, 0.95), (0, 0, 1), (1, 600, 1)):
        rows.run(r.uniform(0, 1, 9), T, k, p).check((T, k, p))
    assert rows.tokens.cpu().flatten().tolist()[1:4] == [-1] * 3
    good = Rows(_logits(r, 4, V), io)
    good.run(0.5, T=[-1, np.nan, np.inf, 1]).check("T")
    assert good.tokens.cpu().flatten().tolist()[:3] == [-1] * 3
    good.run(np.array([np.nan, -2.0, 1.0, 7.5])).check("u")


def test_rejected_drafts():
    """n_reject counts from the first position whose fed token is not the one drawn before it."""
    gu.note("sample rejects")
    r = np.random.default_rng(2)
    B, W, V = 6, 5, 900
    rows = Rows(_logits(r, B * W, V, 1.0), "f32", W=W)
    u = r.uniform(0, 1, (B, W))
    tok = rows.run(u).tokens.cpu().numpy()
    fed = np.zeros((B, W), np.int64)
    fed[:, 1:] = tok[:, :-1]
    for b in range(1, B):        # the first wrong draft at position b (5: none)
        if b < W:
            fed[b, b] = (fed[b, b] + 1) % V
    fed[0, 1] = -1
    rows.run(u, fed=fed).check()
    assert np.array_equal(rows.tokens.cpu().numpy(), tok)
    assert rows.rej.cpu().tolist() == [W - 1, W - 1, W - 2, W - 3, W - 4, 0]
    one = Rows(_logits(r, 3, V), "bf16")
    one.run(0.3, fed=np.zeros((3, 1)))
    assert one.rej.cpu().tolist() == [0, 0, 0]


def test_draws_follow_the_distribution():
    """Even steps of u give each token its share of the draws, to one draw a token."""
    gu.note("sample shares")
    r = np.random.default_rng(9)
    V, n = 11, 4096
    x = np.broadcast_to(r.standard_normal(V), (n, V))
    rows = Rows(x, "f32")
    tok = rows.run((np.arange(n) + 0.5) / n).tokens.cpu().numpy().ravel()
    e = np.exp(rows.x[0] - rows.x[0].max())
    assert np.all(np.abs(np.bincount(tok, minlength=V) - n * e / e.sum()) <= 1.001)
    assert np.all(np.diff(tok) >= 0)


def test_replays_and_streams():
    """A captured call on new logits and random numbers equals the eager one; two calls at once on two streams too."""
    lad = _lad()
    gu.note("sample in a graph")
    r = np.random.default_rng(4)
    B, W, V = 4, 3, 5003
    logits = torch.empty((B, W, V), dtype=torch.bfloat16, device=gu.DEV)
    u, tok = torch.empty((B, W), device=gu.DEV), torch.empty((B, W), dtype=torch.int32, device=gu.DEV)
    fed, rej = torch.zeros((B, W), dtype=torch.int32, device=gu.DEV), torch.empty(B, dtype=torch.int32, device=gu.DEV)
    k, p = _dev(np.array([0, 50, 0, 4500]), torch.int32), _dev(np.array([0.9, 0.9, 1, 0.5], F), torch.float32)
    need = lad.replay_sample_workspace(B, W, V)
    ws = [torch.empty(need, dtype=torch.uint8, device=gu.DEV) if need else None for _ in range(2)]
    logits.copy_(_dev(_logits(r, B * W, V).reshape(B, W, V).astype(F), torch.float32))
    u.uniform_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        lad.replay_sample(logits, u, tok, top_k=k, top_p=p, fed=fed, n_reject=rej, workspace=ws[0])
    for i in range(4):
        logits.copy_(_dev(_logits(r, B * W, V).reshape(B, W, V).astype(F), torch.float32))
        u.uniform_()
        et, er = torch.empty_like(tok), torch.empty_like(rej)
        lad.replay_sample(logits, u, et, top_k=k, top_p=p, fed=fed, n_reject=er, workspace=ws[1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, et) and torch.equal(rej, er), i
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(tok) for _ in range(2)]
    torch.cuda.synchronize()
    for s, o, w in zip(streams, outs, ws):
        lad.replay_sample(logits, u, o, top_k=k, top_p=p, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], et) and torch.equal(outs[1], et)


def test_refusals():
    lad = _lad()
    gu.note("sample refusals")
    x = torch.zeros((2, 3, 100), device=gu.DEV)
    u, tok = torch.zeros((2, 3), device=gu.DEV), torch.zeros((2, 3), dtype=torch.int32, device=gu.DEV)
    rej = torch.zeros(2, dtype=torch.int32, device=gu.DEV)
    for bad in (x.half(), x.cpu(), x.transpose(1, 2), x[:, :, ::2], x[:1].expand(2, 3, 100), torch.zeros((2, 4, 100), device=gu.DEV)[:, :3]):
        with pytest.raises(lad.ReplayError):
            lad.replay_sample(bad, u, tok)
    with pytest.raises(lad.ReplayError, match="status 1"):       # every position the same row
        lad.replay_sample(x[:1, :1].expand(2, 3, 100), u, tok)
    for kw in ({"temperature": u}, {"top_k": torch.zeros(2, device=gu.DEV)}, {"n_reject": rej}, {"fed": tok}):
        with pytest.raises(lad.ReplayError):
            lad.replay_sample(x, u, tok, **kw)
    with pytest.raises(lad.ReplayError, match="status 2"):
        lad.replay_sample(torch.zeros((1, 1, (1 << 18) + 1), device=gu.DEV), u[:1, :1].contiguous(), tok[:1, :1].contiguous())


def test_one_position_rejects_nothing():
    lad = _lad()
    gu.note("sample one position with drafts")
    x = torch.randn(37, 1, 100, device=gu.DEV)
    x[3] = float("nan")
    u = torch.rand(37, 1, device=gu.DEV)
    tokens = torch.empty(37, 1, dtype=torch.int32, device=gu.DEV)
    reject = torch.full((37,), 9, dtype=torch.int32, device=gu.DEV)
    lad.replay_sample(x, u, tokens, fed=torch.zeros_like(tokens), n_reject=reject)
    torch.cuda.synchronize()
    assert bool((reject == 0).all()) and int(tokens[3, 0]) == -1


@pytest.mark.parametrize("io,V", [("bf16", 131072), ("f32", 50021), ("f32", 2049), ("bf16", 20011)])
def test_top_k_past_the_list(io, V):
    """A k of thousands, with and without the other filters; a k that ends among masked tokens, or in a step of many."""
    r = np.random.default_rng(V + 1)
    gu.note(f"sample large k V={V} {io}")
    x = _logits(r, 9, V)
    x[5, r.permutation(V)[:V - V // 8]] = -np.inf      # an eighth is left
    x[6] = np.where(r.uniform(0, 1, V) < 0.3, x[6], -np.inf)
    x[7] = np.round(x[7] * 2) / 2                      # steps of thousands
    x[8, :V // 2] = -1e30                              # half of it beyond the last step
    rows = Rows(x, io)
    n = 9
    for k in (2048, 2049, 2500, V // 3, V // 2 + 7, V - 1):
        for T, p, mp in ((1, 1, 0), (0.7, 0.95, 0), (2.5, 0.999, 0), (1.3, 1, 1e-4), (4, 0.5, 1e-3)):
            rows.run(r.uniform(0, 1, n), T, np.full(n, k), p, mp).check((k, T, p, mp))


@pytest.mark.parametrize("io,V", [("bf16", 20011), ("f32", 20011), ("bf16", 131072)])
def test_rows_that_weigh_almost_nothing(io, V):
    """Top-p, and a k about the number that is left, where nearly all of a row is masked, or far below its largest."""
    r = np.random.default_rng(V + 7)
    gu.note(f"sample mostly masked V={V} {io}")
    x = _logits(r, 6, V)
    left = 60
    for b in range(3):
        x[b, r.permutation(V)[left:]] = -np.inf
    x[3, r.permutation(V)[3000:]] = -np.inf
    x[4] = np.where(r.uniform(0, 1, V) < 0.99, x[4] - 500, x[4])
    rows = Rows(x, io)
    for T, k, p in ((1, 0, 0.98), (0.01, 0, 0.9), (0.1, 0, 0.98), (1, 50, 1), (0.8, left - 1, 0.95), (1, left, 1), (1, left + 1, 0.9),
                    (1, 1000, 1), (0.01, 2500, 0.9), (1, 3500, 0.99), (1, 5000, 0.9)):
        rows.run(r.uniform(0, 1, 6), T, k, p).check((T, k, p))


def test_no_token_matches_no_draft():
    """A position without an answer (token -1) does not stand for a draft of -1, and nothing behind it stays."""
    gu.note("sample -1 against a draft of -1")
    r = np.random.default_rng(6)
    x = _logits(r, 3 * 4, 300)
    x[1], x[4 + 0], x[8 + 2] = np.nan, -np.inf, np.inf
    rows = Rows(x, "f32", W=4)
    tok = rows.run(0.4).tokens.cpu().numpy()
    assert (tok == -1).sum() == 3
    fed = np.full((3, 4), -1)
    fed[:, 1:] = tok[:, :-1]
    rows.run(0.4, fed=fed).check()
    # kept: the position without an answer itself, at most
    assert rows.rej.cpu().tolist() == [2, 3, 1]
