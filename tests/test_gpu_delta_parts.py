"""replay_delta_scan's results as close to float64 as float32 operands leave them,
on every way a prompt can take through the kernels; the limits, and that a part of
an operand less would break them, are test_delta_parts.py's."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from tests import gpu_util as gu
from tests.test_delta_parts import FLIPS, STATE, off
from tests.test_gpu_delta import Prompts, _lad

pytestmark = pytest.mark.gpu


def look(p, seqs, heads):
    """The largest errors over these sequences and heads, state and y of each against its own largest value."""
    torch.cuda.synchronize()
    assert p.err.cpu().eq(0).all()
    H, G, P, N = p.shape
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    groups = [h // (H // G) for h in heads]
    worst, flips = 0.0, []
    for b in seqs:
        rows = p.rows(b)
        x = [f(p.q[rows][:, groups]), f(p.k[rows][:, groups]), f(p.v[rows][:, heads]), f(p.beta[rows][:, heads]),
             f(p.alpha[rows][:, heads])]
        y, S = op.delta_scan(*x, f(p.s_in[b, heads]))
        for i, h in enumerate(heads):
            s, o, d = off(p.y[rows, h].float().cpu().numpy(), p.s_out[b, h].cpu().numpy(), y[:, i], S[i])
            worst = max(worst, s, o if p.io == torch.float32 else 0.0)
            flips.append(d)
    return worst, float(np.mean(flips))


# sequences of these lengths, heads, groups; the way they take with bf16 io
WAYS = [([300, 64, 129], 4, 2, 64, 64),                                # four wavefronts for the state, two for y
        ([300, 40, 129], 4, 2, 64, 128), ([300, 200], 8, 2, 128, 128),
        ([250] * 6, 16, 4, 64, 128), ([250, 64, 190], 16, 4, 128, 128),    # two, and two for y
        ([250] * 10, 16, 4, 64, 64), ([250] * 10, 16, 4, 64, 128), ([250, 300, 64, 65, 190], 16, 4, 128, 128),   # pairs
        ([250, 77], 3, 1, 16, 16)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H,G,P,N", WAYS)
def test_results_hold_their_bits(io, lens, H, G, P, N):
    gu.note(f"delta_scan bits {len(lens)} x {H} heads P={P} N={N} {io}")
    p = Prompts(lens, H, G, P, N, io, first=1, seed=P + N + H)
    p.run()
    worst, flips = look(p, range(len(lens))[:3], [0, H - 1])
    assert worst < STATE, np.log2(worst)
    if io == "bf16":
        assert flips < FLIPS, np.log2(flips)


@pytest.mark.parametrize("lens,H,G,P,N", WAYS)
def test_a_state_that_stays(lens, H, G, P, N):
    """beta 0 and alpha 1: y is S q, and the state keeps every bit."""
    gu.note(f"delta_scan of a state that stays {len(lens)} x {H} heads P={P} N={N}")
    p = Prompts(lens, H, G, P, N, "bf16", seed=P + H, decay=lambda r, s: np.ones(s), beta=lambda r, s: np.zeros(s))
    p.run()
    worst, flips = look(p, range(len(lens))[:3], [0, H - 1])
    assert torch.equal(p.s_out, p.s_in) and flips < FLIPS, np.log2(flips)


def test_over_windows_of_the_workspace():
    """More chunks than the workspace holds at once: the state passes through memory between them."""
    gu.note("delta_scan bits over windows")
    lens = [3000, 1500, 700, 64, 2901, 1, 1000, 2250]
    p = Prompts(lens, 64, 8, 64, 64, "bf16", seed=3)
    chunks = (max(lens) + 63) // 64
    need = [_lad().replay_delta_scan_workspace(p.cfg, p.T, n) for n in (64, max(lens))]
    assert need[1] < chunks * need[0]
    p.run()
    worst, flips = look(p, [0, 4, 7], [0, 63])
    assert worst < STATE and flips < FLIPS, (np.log2(worst), np.log2(flips))
