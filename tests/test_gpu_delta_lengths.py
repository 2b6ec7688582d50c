"""replay_delta_inputs over rows whose squares float32 does not hold.  Bounds as
in test_gpu_delta.py: the squares' sum off by N 2^-24 of itself, three roundings
more, and the io type's; a result of less than 2^-126 by half its least step."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from tests import gpu_util as gu
from tests.test_gpu_delta import E24, _cfg, _dev, _lad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [16, 64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-30, 1e-6, 1e30])
def test_rows_of_any_length(io, N, eps):
    gu.note(f"delta_inputs, rows of any length N={N} eps={eps} {io}")
    P = {16: 16, 64: 64, 128: 128}[N]
    r = np.random.default_rng(N)
    t = torch.bfloat16 if io == "bf16" else torch.float32
    scales = np.array([1e-45, 3e-43, 1e-40, 1e-38, 1e-30, 1e-23, 1e-19, 2.0 ** -41, 2.0 ** -39, 1e-10, 1, 1e10, 1e18, 1e20, 1e30,
                       1e37, 7e37])
    T, H, G = len(scales), 2, 2
    q = _dev(np.clip(r.standard_normal((T, G, N)), -3, 3) * scales[:, None, None], t)
    k = _dev(np.clip(r.standard_normal((T, G, N)), -3, 3) * scales[::-1, None, None], t)
    raw = _dev(r.standard_normal((T, 2 * H)), t)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    beta, alpha = torch.empty(T, H, device=gu.DEV), torch.empty(T, H, device=gu.DEV)
    e32 = float(np.float32(eps))
    _lad().replay_delta_inputs(_cfg(1, H, G, P, N, io), T, q, k, raw[:, :H], raw[:, H:], None, torch.zeros(H, device=gu.DEV), 0.5,
                               eps, qo, ko, beta, alpha)
    torch.cuda.synchronize()
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    e = 2.0 ** -8 if io == "bf16" else E24
    least = 2.0 ** -133 if io == "bf16" else 2.0 ** -149
    with np.errstate(invalid="ignore"):
        for x, got, scale in ((q, qo, 0.5), (k, ko, 1.0)):
            want = op.unit(f(x), e32, scale)
            ok = np.isfinite(want)                      # a zero row with eps 0 has no direction
            err = np.abs(f(got) - want)[ok]
            assert np.all(err <= (((N / 2 + 4) * E24 + e) * np.abs(want) * (1 + 2.0 ** -8) + least)[ok]), float(err.max())
            assert np.isnan(f(got)[~ok]).all()
