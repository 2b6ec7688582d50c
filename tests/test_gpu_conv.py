"""The convolution and discretisation ahead of the recurrence
(replay_conv_prompt, replay_conv_step) against float64.

Bounds, before any run.  A sum of K products and a bias in float32 is off by
at most (K + 1) 2^-24 of the sum of magnitudes m (K + 1 roundings of partial
sums that m bounds; the products are fused); SiLU's slope is below 1.1 and its
exponential, at arguments up to |z|, is good to (|z| + 4) 2^-23, its division
and product to 2^-22 together.  Rounding to the type adds 2^-8 (bf16) or
2^-24 of the result.  dt: the sum raw + bias is off by 2^-24 of itself (slope
at most 1), the three functions by 8 x 2^-24 together; a: A dt by 4 x 2^-24
more (expf of a_log, a product), its own exponential by 4 x 2^-24."""
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


def _cfg(B, H, G, P, N, io, rule=0):
    lad = _lad()
    return lad.ReplayConfig(B, H, G, P, N, 16, lad.BF16 if io == "bf16" else lad.F32, lad.NONE, 0, rule)


class Case:
    """Inputs of one convolution, on the host (float64 views of what the device holds) and on the device."""

    def __init__(self, rows, B, H, G, P, N, io, K, slots, bias=True, pad=0, seed=0, dt_min=0.0, dt_max=float("inf"),
                 act=True):
        r = np.random.default_rng(seed)
        self.io = torch.bfloat16 if io == "bf16" else torch.float32
        self.shape, self.K, self.slots, self.act = (B, H, G, P, N), K, slots, act
        self.C = C = H * P + 2 * G * N
        self.cfg = _cfg(B, H, G, P, N, io)
        # [pad | C channels | H raw step sizes]: an odd pad takes the rows off 16-byte boundaries
        self.wide = torch.from_numpy(r.standard_normal((rows, pad + C + H)).astype(np.float32) * 1.5).to(self.io).to(gu.DEV)
        self.x, self.raw = self.wide[:, pad:pad + C], self.wide[:, pad + C:]
        self.w = r.uniform(-0.7, 0.7, (C, K)).astype(np.float32)
        self.b = r.uniform(-0.5, 0.5, C).astype(np.float32) if bias else None
        self.dt_bias = r.uniform(-5, 1, H).astype(np.float32) if bias else None
        self.a_log = np.log(r.uniform(1, 16, H)).astype(np.float32)
        self.lim = (dt_min, dt_max)
        t = lambda a: None if a is None else torch.from_numpy(a).to(gu.DEV)  # noqa: E731
        self.conv = _lad().ReplayConv(t(self.w), t(self.b), t(self.dt_bias), t(self.a_log), slots=slots, silu=act,
                                      dt_min=dt_min, dt_max=dt_max)
        self.state = torch.from_numpy(r.standard_normal((B, slots, C)).astype(np.float32)).to(self.io).to(gu.DEV)
        self.err = torch.zeros(B + 1, dtype=torch.int32, device=gu.DEV)

    def outs(self, *lead, fill=7.0):
        B, H, G, P, N = self.shape
        mk = lambda *s, dt=self.io: torch.full((*lead, *s), fill, dtype=dt, device=gu.DEV)  # noqa: E731
        return [mk(G, N), mk(G, N), mk(H, P), mk(H, dt=torch.float32), mk(H, dt=torch.float32)]

    def check(self, outs, rows, x, hist):
        """outs: (q, k, v, dt, a) flattened to rows; rows: which rows hold this sequence; x: its float64 rows."""
        B, H, G, P, N = self.shape
        ref, mag, last = op.conv(x, self.w, self.b, hist, self.act)
        flat = [o.reshape(-1, o.shape[-1] if o.dim() == 2 else o.shape[-2] * o.shape[-1])[rows].double().cpu().numpy()
                for o in outs[:3]]
        got = np.concatenate([flat[2], flat[1], flat[0]], 1)
        half = 2.0 ** -8 if self.io == torch.bfloat16 else E24
        z = np.abs(mag)
        tol = 1.1 * (self.K + 1) * E24 * mag + ((z + 4) * 2 * E24 + 4 * E24) * np.abs(ref)
        tol = tol + half * (np.abs(ref) + tol) + 1e-38
        assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
        raw = self.raw[rows].double().cpu().numpy()
        dt, a = op.discretise(raw, self.dt_bias, self.a_log, *self.lim)
        s = np.abs(raw + (0 if self.dt_bias is None else self.dt_bias))
        tdt = (s + 8 * dt) * E24 + 1e-38
        A = np.exp(self.a_log.astype(np.float64))
        ta = a * (A * tdt + 4 * A * dt * E24 + 4 * E24) + 1e-38
        got_dt, got_a = (o.reshape(-1, H)[rows].double().cpu().numpy() for o in outs[3:])
        assert np.all(np.abs(got_dt - dt) <= tdt), float(np.max(np.abs(got_dt - dt) / tdt))
        assert np.all(np.abs(got_a - a) <= ta), float(np.max(np.abs(got_a - a) / ta))
        return last


PROMPTS = [
    # lens, first row, H, G, P, N, io, K, slots, bias, pad, resume
    ([1], 0, 4, 2, 64, 128, "bf16", 4, 3, True, 0, False),
    ([0, 1, 2, 3, 4, 5, 0], 0, 4, 1, 16, 16, "bf16", 4, 3, True, 0, True),
    ([2, 70, 1, 33, 64, 31, 32], 3, 8, 2, 64, 64, "bf16", 4, 9, True, 8, True),
    ([2, 70, 1, 33], 0, 5, 1, 64, 64, "bf16", 4, 4, True, 0, True),        # an odd row: element loads
    ([40, 0, 97], 1, 3, 3, 16, 16, "f32", 4, 3, True, 1, True),
    ([129, 3], 2, 4, 2, 128, 128, "f32", 3, 2, False, 0, True),
    ([5, 66], 0, 4, 4, 64, 128, "f32", 2, 5, True, 0, False),
    ([31, 95], 0, 2, 1, 64, 128, "bf16", 2, 1, False, 3, True),
    ([1000], 0, 128, 8, 64, 128, "bf16", 4, 3, True, 0, True),
]


@pytest.mark.parametrize("lens,first,H,G,P,N,io,K,slots,bias,pad,resume", PROMPTS)
def test_prompt(lens, first, H, G, P, N, io, K, slots, bias, pad, resume):
    B, T = len(lens), first + sum(lens) + 6
    gu.note(f"conv_prompt {lens} H={H} P={P} N={N} {io} K={K} R={slots} pad={pad}")
    c = Case(T, B, H, G, P, N, io, K, slots, bias, pad, seed=sum(lens) + K)
    ends = first + np.cumsum(lens)
    c.wide[:first] = float("nan")            # rows of no sequence are read by none
    c.wide[ends[-1]:] = float("nan")
    cu = torch.tensor([first, *ends], dtype=torch.int32, device=gu.DEV)
    pos = torch.tensor([(5 * b) % 7 + (2 ** 31 - 40 if b % 3 == 2 else 0) for b in range(B)], dtype=torch.int32, device=gu.DEV)
    outs = c.outs(T)
    before = c.state.clone()
    out_state = c.state if resume else torch.full_like(c.state, 3.0)
    kept = out_state.clone()
    _lad().replay_conv_prompt(c.cfg, c.conv, T, cu, c.x, c.raw, pos, c.state if resume else None, out_state, *outs, c.err)
    torch.cuda.synchronize()
    assert c.err.cpu().eq(0).all()
    for o in outs:                            # rows of no sequence are left as they were
        assert bool((o[:first] == 7.0).all()) and bool((o[ends[-1]:] == 7.0).all())
    for b, n in enumerate(lens):
        p, rows = int(pos[b]), slice(int(ends[b]) - n, int(ends[b]))
        slot = [(p - i) % slots for i in range(K - 1, 0, -1)]
        hist = before[b, slot].double().cpu().numpy() if resume else np.zeros((K - 1, c.C))
        last = c.check(outs, rows, c.x[rows].double().cpu().numpy(), hist)
        assert np.array_equal(out_state[b, slot].double().cpu().numpy(), last), b
        rest = [i for i in range(slots) if i not in slot]
        assert torch.equal(out_state[b, rest], kept[b, rest])


def test_prompt_bad_ranges():
    """A decreasing range, one past T, a negative start: flagged, their states left; where the ranges ascend, the
    others are right."""
    lad = _lad()
    gu.note("conv_prompt bad ranges")
    T = 40
    for cu, bad in (([0, 10, 5, 20], [1]), ([0, 10, 20, 50], [2]), ([-3, 8, 8, 20], [0]), ([0, 5, 50, 3], [1, 2])):
        c = Case(T, 3, 4, 2, 16, 16, "bf16", 4, 3, seed=9)
        outs, state = c.outs(T), torch.full_like(c.state, 3.0)
        lad.replay_conv_prompt(c.cfg, c.conv, T, torch.tensor(cu, dtype=torch.int32, device=gu.DEV), c.x, c.raw, None,
                               c.state, state, *outs, c.err)
        torch.cuda.synchronize()
        err = c.err.cpu().tolist()
        assert err[0] == lad.SEQERR_BAD_RANGE
        assert [b for b in range(3) if err[1 + b]] == bad, cu
        for b in range(3):
            if b in bad:
                assert bool((state[b] == 3.0).all())
            elif cu == sorted(cu):
                rows = slice(cu[b], cu[b + 1])
                hist = c.state[b, [(-i) % 3 for i in (3, 2, 1)]].double().cpu().numpy()
                c.check(outs, rows, c.x[rows].double().cpu().numpy(), hist)


@pytest.mark.parametrize("io,pad", [("bf16", 0), ("f32", 0), ("bf16", 5), ("f32", 3)])
@pytest.mark.parametrize("K,W,slots", [(4, 1, 3), (4, 1, 4), (4, 5, 8), (4, 5, 5), (3, 8, 16), (2, 16, 17), (4, 16, 19), (2, 1, 1)])
def test_step(io, pad, K, W, slots):
    lad = _lad()
    B, H, G, P, N = 5, 4, 2, 64, 64
    gu.note(f"conv_step {io} K={K} W={W} R={slots} pad={pad}")
    c = Case(B * W, B, H, G, P, N, io, K, slots, True, pad, seed=K * 100 + W, dt_min=0.002, dt_max=0.9)
    pos = [0, 1, 2 ** 31 - 30, 7, 1000]
    outs, before = c.outs(B, W), c.state.clone()
    lad.replay_conv_step(c.cfg, c.conv, W, c.x, c.raw, torch.tensor(pos, dtype=torch.int32, device=gu.DEV), c.state, *outs)
    torch.cuda.synchronize()
    flat = [o.reshape(B * W, *o.shape[2:]) for o in outs]
    for b in range(B):
        rows = slice(b * W, (b + 1) * W)
        hist = before[b, [(pos[b] - i) % slots for i in range(K - 1, 0, -1)]].double().cpu().numpy()
        c.check(flat, rows, c.x[rows].double().cpu().numpy(), hist)
        new = [(pos[b] + w) % slots for w in range(W)]
        assert torch.equal(c.state[b, new], c.x[rows])
        rest = [i for i in range(slots) if i not in new]
        assert torch.equal(c.state[b, rest], before[b, rest])


@pytest.mark.parametrize("io,pad,K,H", [("bf16", 0, 4, 8), ("bf16", 1, 3, 8), ("f32", 0, 2, 8), ("f32", 3, 4, 8)])
def test_step_of_many_sequences(io, pad, K, H):
    """Enough sequences that a thread takes several, their number no multiple of that; pending rollbacks."""
    lad = _lad()
    B, R = 1030, 5
    gu.note(f"conv_step B={B} {io} pad={pad} K={K}")
    c = Case(B, B, H, 2, 64, 64, io, K, R, True, pad, seed=K)
    r = np.random.default_rng(K)
    pos, base = r.integers(0, 2 ** 31 - 20, B), None
    base, rej = np.maximum(pos - r.integers(0, 4, B), 0), r.integers(-1, 4, B)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=gu.DEV)  # noqa: E731
    outs, before = c.outs(B, 1), c.state.clone()
    lad.replay_conv_step(c.cfg, c.conv, 1, c.x, c.raw, t(pos), c.state, *outs, base=t(base), n_reject=t(rej))
    torch.cuda.synchronize()
    flat = [o.reshape(B, *o.shape[2:]) for o in outs]
    at = np.where((rej >= 0) & (rej <= pos - base), pos - rej, pos)
    for b in [*range(0, B, 97), B - 3, B - 2, B - 1]:
        hist = before[b, [(int(at[b]) - i) % R for i in range(K - 1, 0, -1)]].double().cpu().numpy()
        c.check(flat, slice(b, b + 1), c.x[b:b + 1].double().cpu().numpy(), hist)
    want = before.clone()
    want[torch.arange(B, device=gu.DEV), t(at % R).long()] = c.x
    assert torch.equal(c.state, want)


def test_step_rollback():
    """The tokens follow pos - n_reject where the rollback is in range, pos where it is not."""
    lad = _lad()
    gu.note("conv_step n_reject")
    B, W, K, R = 5, 3, 4, 8
    c = Case(B * W, B, 4, 2, 16, 16, "bf16", K, R, seed=3)
    pos, base, rej = [10, 10, 10, 10, 4], [6, 6, 6, 6, 4], [0, 3, 5, -1, 0]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=gu.DEV)  # noqa: E731
    outs, before, p = c.outs(B, W), c.state.clone(), t(pos)
    lad.replay_conv_step(c.cfg, c.conv, W, c.x, c.raw, p, c.state, *outs, base=t(base), n_reject=t(rej))
    torch.cuda.synchronize()
    assert p.cpu().tolist() == pos
    flat = [o.reshape(B * W, *o.shape[2:]) for o in outs]
    for b, at in enumerate([10, 7, 10, 10, 4]):
        rows = slice(b * W, (b + 1) * W)
        hist = before[b, [(at - i) % R for i in (3, 2, 1)]].double().cpu().numpy()
        c.check(flat, rows, c.x[rows].double().cpu().numpy(), hist)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prompt_then_steps_equal_one_prompt(io):
    """A prompt in two pieces, then tokens one at a time, then windows with rejected drafts: the same bits as the
    whole sequence at once (same sums in the same order)."""
    lad = _lad()
    gu.note(f"conv prompt + steps {io}")
    H, G, P, N, K, R = 4, 2, 64, 128, 4, 8
    c = Case(60, 1, H, G, P, N, io, K, R, seed=11)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=gu.DEV)  # noqa: E731
    whole, st = c.outs(60), torch.zeros_like(c.state)
    lad.replay_conv_prompt(c.cfg, c.conv, 60, t([0, 60]), c.x, c.raw, None, None, st, *whole, c.err)
    st = torch.zeros_like(c.state)
    pos = t([0])
    for lo, hi in ((0, 2), (2, 35)):
        part = c.outs(hi - lo)
        lad.replay_conv_prompt(c.cfg, c.conv, hi - lo, t([0, hi - lo]), c.x[lo:hi], c.raw[lo:hi], pos, st, st, *part, c.err)
        assert all(torch.equal(o, w[lo:hi]) for o, w in zip(part, whole)), (lo, hi)
    at = 35
    for _ in range(4):
        one = c.outs(1, 1)
        lad.replay_conv_step(c.cfg, c.conv, 1, c.x[at:at + 1], c.raw[at:at + 1], pos, st, *one)
        assert all(torch.equal(o[0], w[at:at + 1]) for o, w in zip(one, whole)), at
        pos += 1
        at += 1
    base = t([0])
    for rej in (0, 3, 5, 1):
        five = c.outs(1, 5)
        lad.replay_conv_step(c.cfg, c.conv, 5, c.x[at:at + 5], c.raw[at:at + 5], pos, st, *five)
        assert all(torch.equal(o[0], w[at:at + 5]) for o, w in zip(five, whole)), at
        pos += 5 - rej
        at += 5 - rej
    # a rollback still to come
    pos += 2
    junk = c.outs(1, 2)
    lad.replay_conv_step(c.cfg, c.conv, 2, c.x[:2], c.raw[:2], pos - 2, st, *junk)
    two = c.outs(1, 2)
    lad.replay_conv_step(c.cfg, c.conv, 2, c.x[at:at + 2], c.raw[at:at + 2], pos, st, *two, base=base, n_reject=t([2]))
    assert all(torch.equal(o[0], w[at:at + 2]) for o, w in zip(two, whole))
    assert c.err.cpu().eq(0).all()


def test_extremes():
    """A NaN or infinite row reaches its K - 1 successors and no other sequence; saturated step sizes stay finite."""
    lad = _lad()
    gu.note("conv extremes")
    c = Case(20, 2, 2, 1, 16, 16, "f32", 4, 3, seed=5)
    c.wide[3, 0] = float("nan")
    c.wide[9, 1] = float("inf")
    c.raw[0, 0], c.raw[1, 0], c.raw[2, 0] = 200.0, -200.0, float("nan")
    cu = torch.tensor([0, 10, 20], dtype=torch.int32, device=gu.DEV)
    outs, st = c.outs(20), torch.zeros_like(c.state)
    lad.replay_conv_prompt(c.cfg, c.conv, 20, cu, c.x, c.raw, None, None, st, *outs, c.err)
    torch.cuda.synchronize()
    v = outs[2].reshape(20, -1)
    assert v[3:7, 0].isnan().all() and v[7:, 0].isfinite().all() and v[:3, 0].isfinite().all()
    assert not v[9, 1].isfinite() and v[10:, 1].isfinite().all()
    dt, a = outs[3], outs[4]
    assert abs(float(dt[0, 0]) - (200.0 + float(c.dt_bias[0]))) < 1e-3 and float(a[0, 0]) < 1e-30
    assert float(dt[1, 0]) == 0.0 and float(a[1, 0]) == 1.0
    assert dt[2, 0].isnan() and a[2, 0].isnan()


def test_no_gates_and_gated_delta():
    """Without dt_raw, dt and a are not touched; a Gated DeltaNet layer takes the convolution alone."""
    lad = _lad()
    gu.note("conv without gates")
    c = Case(8, 1, 2, 1, 16, 16, "bf16", 4, 3, seed=6, act=False)
    c.cfg.rule = lad.GATED_DELTA
    cu = torch.tensor([0, 8], dtype=torch.int32, device=gu.DEV)
    outs, st = c.outs(8), torch.zeros_like(c.state)
    with pytest.raises(lad.ReplayError, match="status 2"):
        lad.replay_conv_prompt(c.cfg, c.conv, 8, cu, c.x, c.raw, None, None, st, *outs, c.err)
    lad.replay_conv_prompt(c.cfg, c.conv, 8, cu, c.x, None, None, None, st, *outs, c.err)
    torch.cuda.synchronize()
    assert bool((outs[3] == 7.0).all()) and bool((outs[4] == 7.0).all())
    ref, mag, _ = op.conv(c.x.double().cpu().numpy(), c.w, c.b, np.zeros((3, c.C)), act=False)
    got = torch.cat([outs[2].reshape(8, -1), outs[1].reshape(8, -1), outs[0].reshape(8, -1)], 1).double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 6 * E24 * mag)


def test_graph_replays():
    """A captured step replays on new inputs in the captured buffers, on a stream of its own."""
    lad = _lad()
    gu.note("conv_step in a graph")
    B, W, K, R = 3, 2, 4, 6
    c = Case(B * W, B, 4, 2, 64, 64, "bf16", K, R, seed=21)
    pos = torch.tensor([0, 5, 9], dtype=torch.int32, device=gu.DEV)
    outs = c.outs(B, W)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lad.replay_conv_step(c.cfg, c.conv, W, c.x, c.raw, pos, c.state, *outs)
    for i in range(4):
        c.wide.copy_(torch.randn_like(c.wide.float()).to(c.io))
        eager_state, eager = c.state.clone(), c.outs(B, W)
        lad.replay_conv_step(c.cfg, c.conv, W, c.x, c.raw, pos, eager_state, *eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, e) for o, e in zip(outs, eager)) and torch.equal(c.state, eager_state), i
        pos += W


def test_refusals_of_the_binding():
    lad = _lad()
    gu.note("conv refusals")
    c = Case(6, 2, 4, 2, 16, 16, "bf16", 4, 3, seed=1)
    outs = c.outs(2, 3)
    pos = torch.zeros(2, dtype=torch.int32, device=gu.DEV)
    call = lambda **k: lad.replay_conv_step(c.cfg, k.get("conv", c.conv), 3, k.get("x", c.x), c.raw, k.get("pos", pos),  # noqa: E731
                                            k.get("state", c.state), *k.get("outs", outs))
    for bad in ({"x": c.x.float()}, {"x": c.x[:5]}, {"x": c.x.t()}, {"pos": pos.cpu()}, {"pos": pos.long()},
                {"state": c.state[:, :2]}, {"outs": c.outs(3, 2)}, {"outs": [o.float() for o in outs]}):
        with pytest.raises(lad.ReplayError):
            call(**bad)
    narrow = Case(6, 2, 4, 2, 16, 16, "bf16", 4, 4, seed=1)
    with pytest.raises(lad.ReplayError, match="status 1"):   # a window wider than the state
        lad.replay_conv_step(narrow.cfg, narrow.conv, 5, torch.empty(10, c.C, dtype=c.io, device=gu.DEV), None, pos,
                             narrow.state, *narrow.outs(2, 5))
    call()
    torch.cuda.synchronize()


def test_parameters_of_another_gpu():
    """Taps that lie on another GPU than the current one are refused: the kernels would read them there."""
    import copy
    lad = _lad()
    gu.note("conv parameters of another GPU")
    c = Case(6, 2, 4, 2, 16, 16, "bf16", 4, 3, seed=1)
    pos = torch.zeros(2, dtype=torch.int32, device=gu.DEV)
    other = copy.copy(c.conv)
    other.gpu = c.conv.gpu + 1
    with pytest.raises(lad.ReplayError, match="the current one"):
        lad.replay_conv_step(c.cfg, other, 3, c.x, c.raw, pos, c.state, *c.outs(2, 3))
