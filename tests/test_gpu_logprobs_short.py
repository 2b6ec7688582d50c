"""replay_logprobs where a row, or its last part, has few blocks of logits: fewer
groups of threads with tokens than tokens asked for, with more threads than
that or not.  Bounds as in test_gpu_logprobs.py."""
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_logprobs import Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 9, 20, 32])
@pytest.mark.parametrize("V", [32, 77, 129, 260, 300, 511, 2048 + 40, 2048 + 133, 2458, 8192 + 129, 8192 + 500])
def test_short_parts(io, n, V):
    gu.note(f"logprobs, short part {V} {io} top {n}")
    for B, lead in ((2, 0), (3, 3)):
        p = Rows(B, 2, V, io, 1, n, seed=V + n, lead=lead, pad=1)
        p.run()
        p.check()
    wide = Rows(700, 1, V, io, 0, n, seed=n)   # large parts
    wide.run()
    wide.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [130, 300, 2048 + 200])
def test_equal_and_masked_logits_in_short_parts(io, V):
    gu.note(f"logprobs, equal logits in a short part {V} {io}")
    p = Rows(3, 2, V, io, 1, 32, seed=V)
    p.logits[0] = 1.5
    p.logits[1, :, 5:] = -float("inf")
    p.logits[2, 0, ::2] = torch.finfo(p.t).min
    p.run()
    p.check()
