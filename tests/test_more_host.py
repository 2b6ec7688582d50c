"""What the token score, Gated DeltaNet prompt and draft tree calls refuse on
the host.  No call here reaches the device: every one is rejected before any
launch."""
import ctypes

import pytest

P16 = 0x1000


@pytest.fixture(scope="module")
def lad():
    import linear_attention_decode_amd as m
    return m


def _logprobs(lad, B=2, W=1, V=100, **kw):
    a = dict(logits=P16, dtype=0, stride=V, T=P16, M=1, ids=P16, logp=P16, H=P16, n=3, top=P16, top_lp=P16, ws=P16,
             ws_bytes=1 << 40) | kw
    return lad.lib.replay_logprobs(B, W, V, a["logits"], a["dtype"], a["stride"], a["T"], a["M"], a["ids"], a["logp"], a["H"],
                                   a["n"], a["top"], a["top_lp"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(W=0), 1), (dict(V=0), 1), (dict(V=1 << 18 | 1), 2), (dict(B=1 << 20, W=64), 2), (dict(logits=None), 1),
    (dict(logits=0x1002), 1), (dict(logits=0x1001, dtype=1), 1), (dict(dtype=2), 2), (dict(stride=99), 1), (dict(T=0x1001), 1),
    (dict(M=-1), 1), (dict(ids=None), 1), (dict(logp=None), 1), (dict(ids=0x1002), 1), (dict(H=0x1001), 1), (dict(n=-1), 1),
    (dict(n=33), 2), (dict(n=101), 1), (dict(top=None), 1), (dict(top_lp=None), 1), (dict(top=0x1002), 1), (dict(ws=None), 1),
    (dict(ws=0x1008), 1), (dict(ws_bytes=8), 1),
])
def test_logprobs_refusals(lad, kw, status):
    assert _logprobs(lad, **kw) == status


def test_logprobs_workspace(lad):
    n = ctypes.c_size_t()
    assert lad.lib.replay_logprobs_workspace(1, 1, 100, 5, None) == 1
    assert lad.lib.replay_logprobs_workspace(1, 1, 100, 101, ctypes.byref(n)) == 1
    assert lad.lib.replay_logprobs_workspace(1, 1, 1 << 19, 5, ctypes.byref(n)) == 2
    assert lad.replay_logprobs_workspace(1, 1, 100, 0) > 0
    assert lad.replay_logprobs_workspace(4, 2, 5000, 5) == 8 * lad.replay_logprobs_workspace(1, 1, 5000, 5)
    with pytest.raises(lad.ReplayError):
        lad.replay_logprobs_workspace(1, 1, 1 << 32, 5)
