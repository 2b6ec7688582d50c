"""replay_delta_scan over more chunks than its workspace holds at once (512 MiB):
the same results, window after window, with sequences that end in any of them.
Bounds as in test_gpu_delta.py."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_delta import Prompts, _lad

pytestmark = pytest.mark.gpu


def test_many_sequences_over_three_windows():
    gu.note("delta scan over windows, 64 sequences")
    lens = [int(n) for n in np.random.default_rng(2).integers(1, 600, 64)]
    lens[:8] = [640, 0, 1, 256, 257, 512, 513, 255]
    p = Prompts(lens, 64, 8, 64, 64, "bf16", first=3, seed=8)
    need = _lad().replay_delta_scan_workspace(p.cfg, p.T, 640)
    assert need <= 512 << 20 and _lad().replay_delta_scan_workspace(p.cfg, p.T, 256) == need   # no more than four chunks at once
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.s_out[1], p.s_in[1])
    p.check([0, 2, 3, 4, 5, 6, 7, 63])


@pytest.mark.parametrize("P,N", [(64, 64), (128, 128)])
def test_one_long_prompt_is_its_halves(P, N):
    """Few heads (the chain's other form); cut at a chunk, so the sums' order is the same."""
    gu.note(f"delta scan over windows, one prompt {P}")
    H, G, cut = 100 * 64 // P, 50 * 64 // P, 6400
    n = 64 * (512 << 20 >> 5) // (31488 * H >> 5) // 64 * 64 + 200
    p = Prompts([n], H, G, P, N, "bf16", seed=5, extra=0)
    ws = p.run()
    torch.cuda.synchronize()
    assert ws.numel() * 4 < 31488 * H * (n // 64)   # not all of its chunks
    y, s = p.y.clone(), p.s_out.clone()
    whole, inputs = p.s_in.clone(), (p.q, p.k, p.v, p.beta, p.alpha)
    for a, b in ((0, cut), (cut, n)):
        q = Prompts.__new__(Prompts)
        q.__dict__.update(p.__dict__)
        q.lens, q.T, q.ends, q.s_in = [b - a], b - a, np.array([b - a]), whole
        q.cu = torch.tensor([0, b - a], dtype=torch.int32, device=gu.DEV)
        q.q, q.k, q.v, q.beta, q.alpha = (t[a:b].contiguous() for t in inputs)
        q.y, q.s_out = torch.empty_like(p.y[a:b]), torch.empty_like(s)
        q.run()
        torch.cuda.synchronize()
        assert torch.equal(q.y, y[a:b])
        whole = q.s_out
    assert torch.equal(whole, s) and bool(torch.isfinite(s).all()) and p.err.cpu().eq(0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,H,G,P,N", [([70], 7, 1, 64, 64), ([33, 1, 100], 14, 2, 64, 128), ([64, 65, 3, 0, 130], 26, 2, 64, 64),
                                          ([40, 90], 69, 3, 64, 128), ([129], 36, 1, 128, 128), ([5, 66, 17], 20, 1, 16, 16)])
def test_few_groups(io, lens, H, G, P, N):
    """Groups that several XCDs share, in parts that their heads do not fill."""
    gu.note(f"delta scan, few groups {io} {lens} {H} {G} {P} {N}")
    p = Prompts(lens, H, G, P, N, io, first=2, seed=H + P)
    p.run()
    torch.cuda.synchronize()
    p.check()
