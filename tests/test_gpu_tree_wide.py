"""replay_verify_tree at the widest rows it takes, 2^23 values (31-bit byte
offsets over 64 nodes in float32), and past them."""
import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rule", [0, 1])
def test_widest_rows(rule):
    """The first, a middle and the last heads; bounds as in test_gpu_tree.py."""
    import linear_attention_decode_amd as lad
    gu.note(f"widest tree rows, rule {rule}")
    H, P, N, W, L = 1 << 19, 16, 16, 64, 2
    g = torch.Generator(device=gu.DEV).manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device=gu.DEV)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    layer = lad.ReplayLayer(1, H, 1, P, N, L, io_dtype="f32", rule="gdn" if rule else "mamba2", device=gu.DEV)
    S = randn(1, H, P, N)
    layer.load_checkpoint(S)
    tokens = lambda n: (unit(randn(1, n, 1, N)), unit(randn(1, n, 1, N)), randn(1, n, H, P), torch.rand(1, n, H, generator=g, device=gu.DEV),  # noqa: E731
                        1 - 0.5 * torch.rand(1, n, H, generator=g, device=gu.DEV))
    ring, x = tokens(L), tokens(W)
    layer.append(L, *ring)
    r = np.random.default_rng(1)
    parent = np.array([-1] + [int(r.integers(-1, w)) for w in range(1, W)])
    y = torch.full((1, W, H, P), 7.0, device=gu.DEV)
    layer.verify_tree(W, torch.tensor(parent[None], dtype=torch.int32, device=gu.DEV), *x, y)
    torch.cuda.synchronize()
    assert layer.get_error()[0] == 0
    heads = [0, H // 2 + 5, H - 1]
    cut = lambda ts: [t[0].double().cpu().numpy() for t in (*ts[:2], ts[2][:, :, heads], ts[3][:, :, heads], ts[4][:, :, heads])]  # noqa: E731
    want, mag = ot.verify(parent, W, cut(ring), cut(x), S[0, heads].double().cpu().numpy(), rule)
    tol = (3 * (L + W) + 2 * N + 64) * 2.0 ** -24 * (8 if rule else 1) * mag + 1e-37
    assert np.all(np.abs(y[0][:, heads].double().cpu().numpy() - want) <= tol)
    layer.close()


def test_wider_rows_are_refused():
    import linear_attention_decode_amd as lad
    gu.note("too wide tree rows")
    H, P, N = (1 << 19) + 1, 16, 16
    layer = lad.ReplayLayer(1, H, 1, P, N, 1, io_dtype="bf16", device=gu.DEV)
    e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=gu.DEV)  # noqa: E731
    y = torch.full((1, 1, H, P), 7.0, device=gu.DEV)
    args = (e(1, 1, 1, N), e(1, 1, 1, N), e(1, 1, H, P), e(1, 1, H, t=torch.float32), e(1, 1, H, t=torch.float32), y)
    with pytest.raises(lad.ReplayError, match="(?i)unsupported"):
        layer.verify_tree(1, torch.full((1, 1), -1, dtype=torch.int32, device=gu.DEV), *args)
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
    layer.close()
