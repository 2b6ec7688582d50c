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


def _cfg(lad, **kw):
    c = lad.ReplayConfig(2, 4, 2, 64, 128, 16, lad.BF16, lad.NONE, 0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _delta_inputs(lad, T=8, **kw):
    a = dict(q_in=P16, k_in=P16, b=P16, b_stride=4, a=P16, a_stride=4, bias=P16, a_log=P16, scale=1.0, eps=1e-6, q=P16, k=P16,
             beta=P16, alpha=P16) | kw
    cfg = a.get("cfg") or _cfg(lad, rule=1)
    return lad.lib.replay_delta_inputs(ctypes.byref(cfg), T, a["q_in"], a["k_in"], a["b"], a["b_stride"], a["a"], a["a_stride"],
                                       a["bias"], a["a_log"], a["scale"], a["eps"], a["q"], a["k"], a["beta"], a["alpha"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(q_in=None), 1), (dict(k_in=0x1008), 1), (dict(b=None), 1), (dict(a=0x1001), 1), (dict(b_stride=3), 1),
    (dict(a_stride=3), 1), (dict(bias=0x1002), 1), (dict(a_log=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(k=0x1004), 1), (dict(beta=None), 1), (dict(alpha=0x1001), 1),
])
def test_delta_inputs_refusals(lad, kw, status):
    assert _delta_inputs(lad, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(rule=0), 2), (dict(batch=0), 1), (dict(head_dim=32), 2), (dict(io_dtype=2), 2),
                                       (dict(heads=1 << 12, groups=1 << 12), 2)])
def test_delta_inputs_shapes(lad, kw, status):
    wide = dict(b_stride=1 << 20, a_stride=1 << 20, T=1 << 20)
    assert _delta_inputs(lad, cfg=_cfg(lad, **({"rule": 1} | kw)), **wide) == status
    assert lad.lib.replay_delta_inputs(None, 1, *[P16] * 3, 4, P16, 4, P16, P16, 1.0, 0.0, *[P16] * 4, None) == 1


def _conv(lad, **kw):
    c = lad.ReplayConvParams(4, 8, 1, P16, P16, P16, P16, 0.0, 0.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


C = 4 * 64 + 2 * 2 * 128


def _conv_tree(lad, W=2, cfg=None, conv=None, **kw):
    a = dict(parent=P16, n=P16, x=P16, x_stride=C, raw=P16, raw_stride=4, pos=P16, state=P16, q=P16, k=P16, v=P16, dt=P16, a=P16,
             err=P16) | kw
    cfg, conv = cfg or _cfg(lad), conv or _conv(lad)
    return lad.lib.replay_conv_tree(ctypes.byref(cfg), ctypes.byref(conv), W, a["parent"], a["n"], a["x"], a["x_stride"],
                                    a["raw"], a["raw_stride"], a["pos"], a["state"], a["q"], a["k"], a["v"], a["dt"], a["a"],
                                    a["err"], None)


def _conv_path(lad, W=2, cfg=None, conv=None, **kw):
    a = dict(parent=P16, n=P16, x=P16, x_stride=C, pos=P16, state=P16, err=P16) | kw
    cfg, conv = cfg or _cfg(lad), conv or _conv(lad)
    return lad.lib.replay_conv_path(ctypes.byref(cfg), ctypes.byref(conv), W, a["parent"], a["n"], a["x"], a["x_stride"],
                                    a["pos"], a["state"], a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(W=0), 1), (dict(W=65), 2), (dict(parent=None), 1), (dict(parent=0x1002), 1), (dict(n=0x1001), 1), (dict(x=None), 1),
    (dict(x=0x1001), 1), (dict(x_stride=C - 1), 1), (dict(pos=None), 1), (dict(state=None), 1), (dict(state=0x1008), 1),
    (dict(err=None), 1)])
def test_tree_convolution_refusals(lad, kw, status):
    assert _conv_tree(lad, **kw) == status
    assert _conv_path(lad, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(q=None), 1), (dict(v=0x1008), 1), (dict(dt=None), 1), (dict(a=0x1001), 1),
                                       (dict(raw=0x1001), 1), (dict(raw_stride=3), 1)])
def test_tree_convolution_outputs(lad, kw, status):
    assert _conv_tree(lad, **kw) == status


def test_tree_convolution_structs_and_shapes(lad):
    assert _conv_path(lad, n=None) == 1
    for f in (_conv_tree, _conv_path):
        assert f(lad, conv=_conv(lad, slots=2)) == 1
        assert f(lad, conv=_conv(lad, width=5)) == 2
        assert f(lad, cfg=_cfg(lad, head_dim=32)) == 2
        assert f(lad, cfg=_cfg(lad, heads=3)) == 1
        assert f(lad, cfg=_cfg(lad, batch=1 << 26), W=64) == 2
    assert _conv_tree(lad, cfg=_cfg(lad, rule=1)) == 2           # Gated DeltaNet: no dt_raw


@pytest.mark.parametrize("at,value,status", [
    (0, 0, 1), (1, 0, 1), (1, 65, 2), (2, None, 1), (2, 0x1001, 1), (3, 0x1002, 1), (4, None, 1), (5, 0x1002, 1), (6, None, 1),
    (7, None, 1), (7, 0x1001, 1), (0, 1 << 27, 2)])
def test_accept_tree_refusals(lad, at, value, status):
    args = [2, 4, P16, P16, P16, P16, P16, P16, None]
    args[at] = value
    assert lad.lib.replay_accept_tree(*args) == status


def test_handle_calls_without_a_handle(lad):
    assert lad.lib.replay_verify_tree(None, 4, *[P16] * 8, None) == 1
    assert lad.lib.replay_append_path(None, 4, *[P16] * 7, None) == 1


def _delta_scan(lad, cfg=None, T=64, most=64, **kw):
    a = dict(cu=P16, q=P16, k=P16, v=P16, dt=P16, a=P16, s_in=P16, s_out=0x10000000, y=P16, err=P16, ws=None, ws_bytes=0) | kw
    cfg = cfg or _cfg(lad, rule=1)
    return lad.lib.replay_delta_scan(ctypes.byref(cfg), T, most, a["cu"], a["q"], a["k"], a["v"], a["dt"], a["a"], a["s_in"],
                                     a["s_out"], a["y"], a["err"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(most=0), 1), (dict(cu=None), 1), (dict(cu=0x1002), 1), (dict(q=None), 1), (dict(k=0x1008), 1),
    (dict(v=None), 1), (dict(dt=None), 1), (dict(a=0x1001), 1), (dict(s_in=0x1004), 1), (dict(s_out=None), 1),
    (dict(s_out=P16), 1), (dict(s_out=P16 + 2 * 4 * 64 * 128 * 4 - 16), 1), (dict(y=None), 1), (dict(err=None), 1),
    (dict(T=(1 << 30) + 1), 2),
])
def test_delta_scan_refusals(lad, kw, status):
    assert _delta_scan(lad, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(batch=0), 1), (dict(head_dim=32), 2), (dict(rule=0), 2), (dict(io_dtype=3), 2),
                                       (dict(batch=1 << 20, heads=512), 2), (dict(heads=1 << 19, groups=1 << 19), 2)])
def test_delta_scan_shapes(lad, kw, status):
    cfg = _cfg(lad, **({"rule": 1} | kw))
    assert _delta_scan(lad, cfg=cfg, s_in=None) == status
    n = ctypes.c_size_t()
    assert lad.lib.replay_delta_scan_workspace(ctypes.byref(cfg), 64, 64, ctypes.byref(n)) == status
    assert lad.lib.replay_delta_scan_workspace(ctypes.byref(_cfg(lad, rule=1)), 64, 64, None) == 1
