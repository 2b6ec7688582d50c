"""Gated DeltaNet layers ahead of the ring: their inputs (replay_delta_inputs)
against float64.

Bounds, before any run: a row's squares' sum is off by N 2^-24 of itself, its
root by half that, the quotient and the product by three roundings more, then
one to the io type.  beta: two roundings and the exponential's 2^-22; alpha:
its exponent x by 8 2^-24 of itself (and what the raw sum's rounding makes of
it), the exponential's 2^-22."""
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


def _dev(a, t=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(t).to(gu.DEV)


def _cfg(B, H, G, P, N, io, rule=1):
    lad = _lad()
    return lad.ReplayConfig(B, H, G, P, N, 16, lad.BF16 if io == "bf16" else lad.F32, lad.NONE, 0, rule)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,G,P,N,pad", [(1, 1, 1, 16, 16, 0), (7, 5, 1, 64, 64, 3), (300, 8, 4, 64, 128, 0), (33, 6, 3, 128, 128, 1),
                                           (1001, 2, 2, 16, 16, 5)])
@pytest.mark.parametrize("place", [False, True])
def test_inputs(io, T, H, G, P, N, pad, place):
    gu.note(f"delta_inputs T={T} H={H} G={G} N={N} {io}")
    r = np.random.default_rng(T)
    t = torch.bfloat16 if io == "bf16" else torch.float32
    q, k = _dev(r.standard_normal((T, G, N)), t), _dev(3 * r.standard_normal((T, G, N)), t)
    q[0] = 0.0                                             # no direction: stays zero
    raw = _dev(4 * r.standard_normal((T, 2 * H + pad)), t)
    raw[:, 2 * H:] = float("nan")
    b, a = raw[:, :H], raw[:, H:2 * H]
    bias, a_log = _dev(r.uniform(-4, 1, H)), _dev(np.log(r.uniform(1, 16, H)))
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    eps, scale = 1e-6, N ** -0.5
    want_q, want_k = op.unit(f(q), eps, scale), op.unit(f(k), eps)
    qo, ko = (q, k) if place else (torch.empty_like(q), torch.empty_like(k))
    beta, alpha = torch.empty(T, H, device=gu.DEV), torch.empty(T, H, device=gu.DEV)
    _lad().replay_delta_inputs(_cfg(1, H, G, P, N, io), T, q, k, b, a, bias, a_log, scale, eps, qo, ko, beta, alpha)
    torch.cuda.synchronize()
    e = 2.0 ** -8 if io == "bf16" else E24
    for got, want in ((qo, want_q), (ko, want_k)):
        assert np.all(np.abs(f(got) - want) <= ((N / 2 + 4) * E24 + e) * np.abs(want) * (1 + 2.0 ** -8) + 1e-37)
    wb, wa = op.delta_gates(f(b), f(a), f(bias), f(a_log))
    assert np.all(np.abs(f(beta) - wb) <= 8 * E24 * wb)
    step = np.logaddexp(f(a) + f(bias), 0)
    x = np.exp(f(a_log)) * step
    off = (8 * x + 2 * np.exp(f(a_log)) * (np.abs(f(a)) + np.abs(f(bias)))) * E24 + 4 * E24
    assert np.all(np.abs(f(alpha) - wa) <= off * wa + 1e-37)


def test_inputs_without_bias_and_with_values_that_are_no_numbers():
    """A row with a NaN is NaN, its neighbours are not; gates at their ends."""
    gu.note("delta_inputs specials")
    T, H, G, N = 4, 2, 2, 64
    q, k = torch.randn(T, G, N, device=gu.DEV), torch.randn(T, G, N, device=gu.DEV)
    q[1, 1, 5] = float("nan")
    inf = float("inf")
    b = torch.tensor([[-inf, inf], [0, -200], [200, float("nan")], [1, 2]], device=gu.DEV)
    a = torch.tensor([[-inf, inf], [0, -200], [200, float("nan")], [1, 2]], device=gu.DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    beta, alpha = torch.empty(T, H, device=gu.DEV), torch.empty(T, H, device=gu.DEV)
    _lad().replay_delta_inputs(_cfg(1, H, G, 64, N, "f32"), T, q, k, b, a, None, torch.zeros(H, device=gu.DEV), 1.0, 0.0, qo, ko,
                               beta, alpha)
    nan = torch.isnan(qo)
    assert nan[1, 1].all() and int(nan.sum()) == N and not torch.isnan(ko).any()
    assert beta.cpu()[:2].tolist() == [[0.0, 1.0], [0.5, 0.0]] and float(beta[2, 0]) == 1.0 and bool(torch.isnan(beta[2, 1]))
    assert alpha.cpu()[0].tolist() == [1.0, 0.0] and alpha.cpu()[1].tolist() == [0.5, 1.0]
    assert float(alpha[2, 0]) == 0.0 and bool(torch.isnan(alpha[2, 1]))
