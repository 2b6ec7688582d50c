"""The gated delta rule with beta up to 2, where I - beta k k^T turns a key's direction
round: prompts and trees against float64, with the bounds of test_gpu_delta.py and
test_gpu_tree.py, which need no more than that the erasure lengthens no row (|1 - beta| <= 1)."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from tests import gpu_util as gu
from tests.test_gpu_delta import SHAPES, Prompts, _dev
from tests.test_gpu_tree import Round

pytestmark = pytest.mark.gpu
BETAS = {"between": lambda r, s: r.uniform(1, 2, s), "two": lambda r, s: np.full(s, 2.0),
         "any": lambda r, s: r.choice([0.0, 1.0, 2.0, 1.5, 0.5], s)}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("beta", sorted(BETAS))
@pytest.mark.parametrize("like", [0.0, 3.0])
def test_prompts(io, P, N, beta, like):
    gu.note(f"delta_scan beta {beta} like {like} P={P} N={N} {io}")
    p = Prompts([400, 77, 64], 4, 2, P, N, io, seed=int(P + like), decay=lambda r, s: np.exp(-r.uniform(0, 1e-3, s)), like=like,
                beta=BETAS[beta])
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("P,N,B,H", [(64, 64, 12, 16), (64, 128, 12, 16), (128, 128, 6, 16), (64, 128, 6, 16)])
def test_prompts_of_many_heads(P, N, B, H):
    """The ways that many sequences and heads take with bf16 io."""
    gu.note(f"delta_scan beta 2, {B} x {H} heads P={P} N={N}")
    p = Prompts([150 + 7 * b for b in range(B)], H, 4, P, N, "bf16", seed=B, decay=lambda r, s: np.exp(-r.uniform(0, 1e-2, s)), like=1.0,
                beta=BETAS["any"])
    p.run()
    torch.cuda.synchronize()
    p.check([0, B - 1])


class Turned(Round):
    """Nodes and ring entries with such betas, keys that share a direction, decays near one."""
    beta, like = "two", 3.0

    def tokens(self, W):
        q, k, v, _, _ = super().tokens(W)
        r, (B, H, G, P, N) = self.r, self.shape
        if not hasattr(self, "shared"):
            self.shared = r.standard_normal((1, 1, G, N))
        k = op.unit(r.standard_normal((B, W, G, N)) + self.like * self.shared, 0)
        return q, _dev(k, self.io), v, _dev(BETAS[self.beta](r, (B, W, H))), _dev(np.exp(-r.uniform(0, 1e-2, (B, W, H))))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("beta", sorted(BETAS))
@pytest.mark.parametrize("shape", ["chain", "random"])
def test_trees(io, P, N, beta, shape):
    gu.note(f"tree beta {beta} {shape} P={P} N={N} {io}")
    cls = type("T", (Turned,), {"beta": beta})
    W = 40
    p = cls(2, 4, 2, P, N, 16, W, io, 1, seed=P, counts=[16, 3], parent=[np.arange(W) - 1] * 2 if shape == "chain" else None)
    p.run()
    p.check()
