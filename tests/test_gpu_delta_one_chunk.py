"""replay_delta_scan where a single chunk of every sequence and head is more than 512
MiB: the workspace is that chunk, used again for each.  Bounds as in test_gpu_delta.py
and test_gpu_delta_parts.py."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from tests.test_delta_parts import FLIPS, STATE
from tests.test_gpu_delta import Prompts, _lad
from tests.test_gpu_delta_parts import look

pytestmark = pytest.mark.gpu


def test_a_chunk_at_a_time():
    gu.note("delta_scan, a chunk of 14720 heads at a time")
    B, H = 230, 64
    lens = [int(n) for n in np.random.default_rng(1).integers(1, 200, B)]
    lens[:6] = [199, 0, 64, 65, 128, 1]
    p = Prompts(lens, H, 8, 64, 64, "bf16", first=2, seed=9)
    need = [_lad().replay_delta_scan_workspace(p.cfg, p.T, n) for n in (1, 64, 65, 200)]
    assert need == [37632 * B * H] * 4 and need[0] > 512 << 20
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.s_out[1], p.s_in[1])
    p.check([0, 2, 3, 4, 5, B - 1])
    worst, flips = look(p, [0, 3, 4], [0, H - 1])
    assert worst < STATE and flips < FLIPS, (np.log2(worst), np.log2(flips))
