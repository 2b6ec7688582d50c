"""Log-probabilities, entropy and top alternatives (replay_logprobs) against float64.

Bounds, before any run: an exponent t = (m - x) / T is off by three roundings,
3 t 2^-24, its exponential by 2^-21 of itself beside that, a block's sum of up
to 8 by 3 2^-24; e^-t t <= 1, so Z - 1 is off by at most (8 + 3 + 3) 2^-24 of
itself plus 3 2^-24 of e^-t t, whose sum is the spread S = sum e^-t t, and
log Z by that over Z; the entropy's own sum by (14 + 3 t) 2^-24 of each term.
A result is then rounded to float32.  Terms below 2^-126, which the float32
exponential does not hold, count as nothing: up to V 2^-126 less in Z, and V
126 ln 2 2^-126 in S (t e^-t falls from t = 1 on)."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24


def _lad():
    import linear_attention_decode_amd as lad
    return lad


def reference(x, T):
    """One row in float64: (log p, entropy, their bounds, the order), or None where it has no distribution."""
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all() or not 0 <= T < np.inf:
        return None
    order = np.argsort(-x, kind="stable")
    if T == 0:
        lp = np.where(np.arange(len(x)) == order[0], 0.0, -np.inf)
        return lp, 0.0, np.zeros(len(x)), 0.0, order
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        t = (x.max() - x) / T
        e = np.exp(-t)
        te = np.where(e > 0, t * e, 0.0)
        tte = np.where(e > 0, t * te, 0.0)
    rest = np.delete(e, order[0]).sum()     # not e.sum() - 1, which float64 takes to 2^-53 of 1, not of itself
    Z, S = 1 + rest, te.sum()
    log_z = np.log1p(rest)
    off_z = (14 * rest + 3 * S) * E24 / Z + len(x) * 2.0 ** -126
    off_h = off_z + ((14 * S + 3 * tte.sum()) * E24 + S / Z * (14 * rest + 3 * S) * E24) / Z
    lp, H = -t - log_z, log_z + S / Z
    return lp, H, off_z + 2 * E24 * np.where(np.isfinite(lp), np.abs(lp), 0), off_h + 2 * E24 * H + len(x) * 88 * 2.0 ** -126, order


class Rows:
    def __init__(self, B, W, V, io, M, n, seed=0, spread=2.2, temperature=None, pad=0, lead=0):
        r = np.random.default_rng(seed)
        x = r.standard_normal((B, W, V)) * spread
        self.t = torch.float32 if io == "f32" else torch.bfloat16
        wide = torch.full((B, W, lead + V + pad), float("nan"), dtype=self.t, device=gu.DEV)
        wide[..., lead:lead + V] = torch.from_numpy(x).to(self.t).to(gu.DEV)
        self.logits = wide[..., lead:lead + V]
        self.T = temperature
        self.ids = torch.from_numpy(r.integers(0, V, (B, W, M)).astype(np.int32)).to(gu.DEV) if M else None
        self.shape, self.M, self.n = (B, W, V), M, n

    def run(self, stream=None, ws=None):
        B, W, V = self.shape
        full = lambda *s, v=7.0, t=torch.float32: torch.full(s, v, dtype=t, device=gu.DEV)  # noqa: E731
        self.logp = full(B, W, self.M) if self.M else None
        self.H = full(B, W)
        self.top = full(B, W, self.n, v=-7, t=torch.int32) if self.n else None
        self.top_lp = full(B, W, self.n) if self.n else None
        if ws is None:
            ws = full(_lad().replay_logprobs_workspace(B, W, V, self.n) // 4, v=float("nan"))
        T = None if self.T is None else torch.tensor(self.T, dtype=torch.float32, device=gu.DEV)
        _lad().replay_logprobs(self.logits, self.ids, self.logp, self.H, self.top, self.top_lp, T, ws, stream)

    def check(self):
        torch.cuda.synchronize()
        B, W, V = self.shape
        x = self.logits.double().cpu().numpy()
        H = self.H.double().cpu().numpy()
        for b in range(B):
            T = 1.0 if self.T is None else float(np.float32(self.T[b]))
            for w in range(W):
                ref = reference(x[b, w], T)
                if ref is None:
                    assert np.isnan(H[b, w])
                    assert self.ids is None or bool(torch.isnan(self.logp[b, w]).all())
                    assert self.top is None or (self.top[b, w].eq(-1).all() and torch.isnan(self.top_lp[b, w]).all())
                    continue
                lp, h, off, off_h, order = ref
                assert abs(H[b, w] - h) <= off_h + 1e-37, (b, w, H[b, w], h, off_h)

                def near(got, at):
                    got, want, tol = got.double().cpu().numpy(), lp[at], off[at]
                    with np.errstate(invalid="ignore"):
                        same = (got == want) | (np.abs(got - want) <= tol + 1e-37)
                    assert same.all(), (b, w, got[~same], want[~same], tol[~same])
                if self.ids is not None:
                    ids = self.ids[b, w].cpu().numpy()
                    good = (ids >= 0) & (ids < V)
                    assert bool(torch.isnan(self.logp[b, w].cpu()[~torch.from_numpy(good)]).all())
                    near(self.logp[b, w].cpu()[torch.from_numpy(good)], ids[good])
                if self.top is not None:
                    assert self.top[b, w].cpu().tolist() == order[:self.n].tolist()
                    near(self.top_lp[b, w], order[:self.n])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,W,V,M,n", [
    (1, 1, 1, 1, 1), (2, 1, 2, 2, 2), (3, 2, 33, 1, 32), (2, 3, 255, 3, 5), (1, 1, 2041, 1, 8), (2, 2, 2048, 0, 20),
    (1, 2, 8191, 5, 32), (1, 1, 50021, 1, 0), (2, 1, 131072, 1, 20), (1, 1, 262144, 2, 32), (40, 4, 60001, 1, 7),
    (3, 400, 777, 1, 3)])
def test_rows(io, B, W, V, M, n):
    gu.note(f"logprobs {B}x{W} V={V} {io} given {M} top {n}")
    p = Rows(B, W, V, io, M, n, seed=V + n)
    p.run()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pad,lead", [(1, 0), (3, 1), (5, 7), (13, 2)])
def test_rows_off_their_alignment(io, pad, lead):
    """Rows of any stride, from any element on; what lies between them is NaN."""
    gu.note(f"logprobs stride {pad} {lead} {io}")
    p = Rows(3, 2, 4099, io, 2, 9, seed=pad, pad=pad, lead=lead)
    p.run()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0.0, 1e-3, 0.3, 1.0, 50.0, 1e30, float("inf"), -1.0, float("nan")])
def test_temperatures(io, T):
    gu.note(f"logprobs T={T} {io}")
    p = Rows(2, 2, 3001, io, 3, 6, seed=5, temperature=[T, 0.8])
    p.ids[:, :, 0] = p.logits.float().argmax(-1).int()
    p.run()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 20, 32])
@pytest.mark.parametrize("V", [40, 3000, 70001])
def test_equal_logits(io, V, n):
    """All equal: more tokens from the bound on than can be gathered; and a few values, many times each."""
    gu.note(f"logprobs equal V={V} n={n} {io}")
    p = Rows(4, 1, V, io, 1, n)
    p.logits[0] = 1.5
    p.logits[1] = torch.randint(0, 3, (1, V), device=gu.DEV).to(p.t)
    p.logits[2] = 0.0
    p.logits[2, 0, 1::2] = -0.0
    p.logits[3] = -float("inf")
    p.logits[3, 0, V // 2:V // 2 + 3] = 2.0      # then the -infinities by index
    p.run()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_values_that_are_no_numbers(io):
    """A NaN, +infinity or -infinities alone: no distribution, for that row; -infinities among others weigh nothing."""
    gu.note(f"logprobs specials {io}")
    p = Rows(6, 1, 9001, io, 4, 5, seed=2)
    inf = float("inf")
    p.logits[0, 0, 8999] = float("nan")
    p.logits[1, 0, 0] = inf
    p.logits[2] = -inf
    p.logits[3, 0, ::2] = -inf
    p.logits[4, 0, :] = torch.finfo(p.t).min     # the type's lowest value everywhere but at one token
    p.logits[4, 0, 77] = 3.0
    p.ids[:, 0, 0] = -1
    p.ids[:, 0, 1] = 9001
    p.ids[:, 0, 2] = 77
    p.run()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_one_token_holds_nearly_all(io):
    """Its log-probability is what the others leave: a small number, to its own bits."""
    gu.note(f"logprobs nearly one {io}")
    p = Rows(2, 1, 5000, io, 1, 3, seed=3, spread=1.0)
    p.logits[0, 0, 1234] = 40.0
    p.logits[1, 0, 4321] = 90.0
    p.ids[0], p.ids[1] = 1234, 4321
    p.run()
    p.check()
    assert float(p.logp[0]) < 0


def test_graph_replays():
    """A captured call serves new logits, given tokens and temperatures; eager work runs between the replays."""
    gu.note("logprobs graph")
    p = Rows(3, 2, 40001, "bf16", 2, 10, seed=1, temperature=[0.5, 1.0, 0.0])
    B, W, V = p.shape
    ws = torch.empty(_lad().replay_logprobs_workspace(B, W, V, 10), dtype=torch.uint8, device=gu.DEV)
    T = torch.tensor(p.T, device=gu.DEV)
    p.run(ws=ws)

    def call():
        _lad().replay_logprobs(p.logits, p.ids, p.logp, p.H, p.top, p.top_lp, T, ws)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        q = Rows(B, W, V, "bf16", 2, 10, seed=10 + i, temperature=[0.3 + i, 0.0, 2.0])
        p.logits.copy_(q.logits)
        p.ids.copy_(q.ids)
        T.copy_(torch.tensor(q.T, device=gu.DEV))
        p.T = q.T
        p.H.fill_(7.0)
        p.top.fill_(-7)
        g.replay()
        p.check()
        (p.logits.float() * 2).sum().item()


def test_refusals_of_the_binding():
    lad = _lad()
    p = Rows(2, 2, 100, "f32", 1, 3)
    ws = torch.empty(lad.replay_logprobs_workspace(2, 2, 100, 3), dtype=torch.uint8, device=gu.DEV)
    f = lambda *s: torch.empty(*s, device=gu.DEV)  # noqa: E731
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device=gu.DEV)  # noqa: E731
    for bad in (dict(ids=i(2, 2, 1)), dict(logp=f(2, 2, 1)), dict(top_ids=i(2, 2, 3)), dict(ids=i(2, 2), logp=f(2, 2)),
                dict(ids=i(2, 2, 2), logp=f(2, 2, 1)), dict(entropy=f(4)), dict(top_ids=f(2, 2, 3), top_logp=f(2, 2, 3)),
                dict(temperature=f(3)), dict(top_ids=i(2, 2, 33), top_logp=f(2, 2, 33)), dict(workspace=ws[1:]),
                dict(workspace=ws[:112]), dict(workspace=None), dict(entropy=torch.empty(2, 2))):
        with pytest.raises(lad.ReplayError):
            lad.replay_logprobs(p.logits, **({"workspace": ws, "entropy": f(2, 2)} | bad))
    with pytest.raises(lad.ReplayError):
        lad.replay_logprobs(p.logits[:, :, ::2], entropy=f(2, 2), workspace=ws)
    with pytest.raises(lad.ReplayError):
        lad.replay_logprobs(p.logits.half(), entropy=f(2, 2), workspace=ws)
