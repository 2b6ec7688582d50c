"""replay_logprobs where the distance of two finite logits is past float32's
range and the temperature brings it back; bounds as in test_gpu_logprobs.py."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_logprobs import Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V,n", [(4, 2), (300, 5), (50021, 20)])
def test_distances_past_the_range(io, V, n):
    gu.note(f"logprobs, far logits V={V} {io}")
    p = Rows(3, 2, V, io, 3, n, seed=V, temperature=[3e38, 1e37, 5e36])
    x = np.random.default_rng(V).uniform(-3.3e38, 3.3e38, (3, 2, V))
    x[..., 0], x[..., 1] = -3.3e38, 3.3e38
    p.logits.copy_(torch.from_numpy(x))
    p.run()
    p.check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_smallest_logits_and_temperatures(io):
    """Logits that differ by the least numbers of their type, temperatures of their size."""
    gu.note(f"logprobs, small logits {io}")
    p = Rows(3, 1, 40, io, 2, 4, seed=1, temperature=[1e-38, 3e-40, 2.0])
    r = np.random.default_rng(2)
    step = 2.0 ** -149 if io == "f32" else 2.0 ** -133
    p.logits.copy_(torch.from_numpy(r.integers(-3, 4, (3, 1, 40)) * step))
    p.logits[0] = torch.from_numpy(r.uniform(-3e-38, 3e-38, (1, 40))).to(p.logits)
    p.run()
    p.check()
