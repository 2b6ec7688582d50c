"""What the prompt, token-input and sampling calls refuse on the host.  No
call here reaches the device: every one is rejected before any launch."""
import ctypes

import pytest

P16 = 0x1000


@pytest.fixture(scope="module")
def lad():
    import linear_attention_decode_amd as m
    return m


def _cfg(lad, **kw):
    c = lad.ReplayConfig(2, 4, 2, 64, 128, 16, lad.BF16, lad.NONE, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _conv(lad, **kw):
    c = lad.ReplayConvParams(4, 8, 1, P16, P16, P16, P16, 0.0, 0.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


C = 4 * 64 + 2 * 2 * 128


def _prompt(lad, cfg=None, conv=None, T=8, **kw):
    a = dict(cu=P16, x=P16, x_stride=C, raw=P16, raw_stride=4, pos=P16, state_in=P16, state_out=P16, q=P16, k=P16, v=P16,
             dt=P16, a=P16, err=P16) | kw
    cfg, conv = cfg or _cfg(lad), conv or _conv(lad)
    return lad.lib.replay_conv_prompt(ctypes.byref(cfg), ctypes.byref(conv), T, a["cu"], a["x"], a["x_stride"], a["raw"],
                                      a["raw_stride"], a["pos"], a["state_in"], a["state_out"], a["q"], a["k"], a["v"],
                                      a["dt"], a["a"], a["err"], None)


def _step(lad, cfg=None, conv=None, W=2, **kw):
    a = dict(x=P16, x_stride=C, raw=P16, raw_stride=4, pos=P16, base=P16, rej=P16, state=P16, q=P16, k=P16, v=P16, dt=P16,
             a=P16) | kw
    cfg, conv = cfg or _cfg(lad), conv or _conv(lad)
    return lad.lib.replay_conv_step(ctypes.byref(cfg), ctypes.byref(conv), W, a["x"], a["x_stride"], a["raw"],
                                    a["raw_stride"], a["pos"], a["base"], a["rej"], a["state"], a["q"], a["k"], a["v"],
                                    a["dt"], a["a"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), 1), (dict(x=None), 1), (dict(x=0x1001), 1), (dict(x_stride=C - 1), 1), (dict(raw=0x1001), 1),
    (dict(raw_stride=3), 1), (dict(pos=0x1002), 1), (dict(state_in=0x1008), 1), (dict(state_out=None), 1),
    (dict(state_out=0x1004), 1), (dict(q=None), 1), (dict(k=0x1008), 1), (dict(v=None), 1), (dict(dt=None), 1),
    (dict(a=None), 1), (dict(err=None), 1), (dict(T=0), 1), (dict(T=-5), 1),
])
def test_prompt_convolution_refusals(lad, kw, status):
    assert _prompt(lad, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(x_stride=C - 1), 1), (dict(pos=None), 1), (dict(base=None), 1), (dict(rej=0x1001), 1),
    (dict(state=None), 1), (dict(state=0x1008), 1), (dict(W=0), 1), (dict(W=17), 1), (dict(W=9), 1), (dict(q=0x1002), 1),
])
def test_token_convolution_refusals(lad, kw, status):
    assert _step(lad, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(width=1), 1), (dict(width=5), 2), (dict(slots=2), 1), (dict(silu=2), 1), (dict(weight=None), 1),
    (dict(weight=0x1002), 1), (dict(bias=0x1001), 1), (dict(a_log=None), 1), (dict(dt_min=-1.0), 1),
    (dict(dt_min=0.5, dt_max=0.1), 1), (dict(dt_min=float("nan")), 1),
])
def test_convolution_parameters(lad, kw, status):
    assert _prompt(lad, conv=_conv(lad, **kw)) == status
    assert _step(lad, conv=_conv(lad, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(heads=3), 1), (dict(head_dim=32), 2), (dict(io_dtype=2), 2), (dict(rule=2), 1),
    (dict(rule=1), 2),                               # Gated DeltaNet: no dt_raw
    (dict(heads=1 << 20, groups=1 << 18), 2),       # channels past 2^24
])
def test_convolution_shapes(lad, kw, status):
    wide = dict(x_stride=1 << 30, raw_stride=1 << 30)
    assert _prompt(lad, cfg=_cfg(lad, **kw), **wide) == status
    assert _step(lad, cfg=_cfg(lad, **kw), **wide) == status


def test_null_structs(lad):
    assert lad.lib.replay_conv_prompt(None, None, 8, *([P16, P16, C, P16, 4] + [P16] * 10)) == 1
    cfg = _cfg(lad)
    assert lad.lib.replay_conv_step(ctypes.byref(cfg), None, 1, P16, C, P16, 4, *([P16] * 9), None) == 1


def _scan(lad, cfg=None, T=64, most=64, **kw):
    a = dict(cu=P16, q=P16, k=P16, v=P16, dt=P16, a=P16, s_in=P16, s_out=0x10000000, y=P16, err=P16, ws=None, ws_bytes=0) | kw
    cfg = cfg or _cfg(lad)
    return lad.lib.replay_scan(ctypes.byref(cfg), T, most, a["cu"], a["q"], a["k"], a["v"], a["dt"], a["a"], a["s_in"],
                               a["s_out"], a["y"], a["err"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(most=0), 1), (dict(cu=None), 1), (dict(cu=0x1002), 1), (dict(q=None), 1), (dict(k=0x1008), 1),
    (dict(v=None), 1), (dict(dt=None), 1), (dict(a=0x1001), 1), (dict(s_in=0x1004), 1), (dict(s_out=None), 1),
    (dict(s_out=P16), 1),                            # in place
    (dict(s_out=P16 + 2 * 4 * 64 * 128 * 4 - 16), 1),   # the last bytes of s_in
    (dict(y=None), 1), (dict(err=None), 1),
    (dict(T=4096, most=4096), 1),                    # segments without their workspace
    (dict(T=4096, most=4096, ws=0x1008, ws_bytes=1 << 40), 1),
])
def test_scan_refusals(lad, kw, status):
    assert _scan(lad, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(batch=0), 1), (dict(head_dim=32), 2), (dict(rule=1), 2), (dict(io_dtype=3), 2),
                                       (dict(batch=1 << 20, heads=512), 2)])
def test_scan_shapes(lad, kw, status):
    assert _scan(lad, cfg=_cfg(lad, **kw), s_in=None) == status
    n = ctypes.c_size_t()
    assert lad.lib.replay_scan_workspace(ctypes.byref(_cfg(lad, **kw)), 64, 64, ctypes.byref(n)) == status


def test_scan_workspace(lad):
    """None where the (sequence, head) pairs fill the GPU or the prompts are short; whole states and decays otherwise."""
    assert lad.replay_scan_workspace(_cfg(lad, batch=64, heads=128), 64 * 4096, 4096) == 0
    assert lad.replay_scan_workspace(_cfg(lad, batch=1, heads=4), 200, 200) == 0
    n = lad.replay_scan_workspace(_cfg(lad, batch=1, heads=8), 8192, 8192)
    assert n > 0 and n % (8 * (64 * 128 + 1) * 4) == 0
    assert lad.replay_scan_workspace(_cfg(lad, batch=1, heads=8), 8192, 1 << 30) == n    # no sequence is longer than T
    for args in ((0, 8), (8, 0)):
        with pytest.raises(lad.ReplayError, match="status 1"):
            lad.replay_scan_workspace(_cfg(lad), *args)


def _sample(lad, B=2, W=3, V=100, **kw):
    a = dict(logits=P16, dtype=lad.BF16, stride=V, opt=lad.ReplaySampling(P16, P16, P16, P16), u=P16, tokens=P16, probs=P16,
             fed=P16, rej=P16, ws=None, ws_bytes=0) | kw
    opt = None if a["opt"] is None else ctypes.byref(a["opt"])
    return lad.lib.replay_sample(B, W, V, a["logits"], a["dtype"], a["stride"], opt, a["u"], a["tokens"], a["probs"], a["fed"],
                                 a["rej"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(W=0), 1), (dict(V=0), 1), (dict(V=(1 << 18) + 1), 2), (dict(B=1 << 20, W=1 << 12), 2),
    (dict(dtype=2), 2), (dict(dtype=-1), 2), (dict(logits=None), 1), (dict(logits=0x1001), 1), (dict(stride=99), 1),
    (dict(u=None), 1), (dict(u=0x1002), 1), (dict(tokens=None), 1), (dict(probs=0x1001), 1), (dict(fed=None), 1),
    (dict(rej=None), 1),
])
def test_sample_refusals(lad, kw, status):
    assert _sample(lad, **kw) == status


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p"])
def test_sample_settings_refusals(lad, name):
    opt = lad.ReplaySampling(P16, P16, P16, P16)
    setattr(opt, name, 0x1001)
    assert _sample(lad, opt=opt) == 1
    n = ctypes.c_size_t()
    assert lad.lib.replay_sample_workspace(0, 1, 1, ctypes.byref(n)) == 1
    assert lad.lib.replay_sample_workspace(1, 1, 1, None) == 1


@pytest.mark.parametrize("io", [0, 1])
def test_scan_limits(lad, io):
    """Rows that a chunk's 32-bit offsets do not reach, tokens an int does not count, workgroups a launch does not number."""
    for kw, T in ((dict(heads=1 << 18, groups=2), 64), (dict(heads=1 << 18, groups=1 << 18), 64),
                  (dict(batch=1, heads=2), (1 << 30) + 1), (dict(batch=1 << 20, heads=64), 64)):
        cfg, n = _cfg(lad, io_dtype=io, **kw), ctypes.c_size_t()
        if T == 64 and "batch" not in kw:
            cfg.heads = cfg.heads * 2          # H P = 2^25
        assert _scan(lad, cfg=cfg, T=T, most=T, s_in=None) == 2, kw
        assert lad.lib.replay_scan_workspace(ctypes.byref(cfg), T, T, ctypes.byref(n)) == 2, kw
    n = ctypes.c_size_t()
    assert lad.lib.replay_scan_workspace(ctypes.byref(_cfg(lad, io_dtype=io, batch=1, heads=2)), 1 << 30, 1 << 30,
                                         ctypes.byref(n)) == 0


def test_launch_limits(lad):
    """More workgroups than a launch numbers (its threads in 32 bits)."""
    assert _prompt(lad, T=(1 << 31) - 1) == 2
    assert _step(lad, cfg=_cfg(lad, batch=1 << 27), W=8) == 2
    assert _sample(lad, B=1 << 23, W=1) == 2
    n = ctypes.c_size_t()
    assert lad.lib.replay_sample_workspace(1 << 22, 2, 8, ctypes.byref(n)) == 2
    assert lad.lib.replay_sample_workspace((1 << 23) - 1, 1, 8, ctypes.byref(n)) == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("P,N", [(16, 16), (64, 64), (64, 128), (128, 128)])
def test_no_scan_in_two_segments(lad, io, P, N):
    """Two segments take two passes over a half: three are the fewest that a plan may have."""
    for heads in (1, 2, 7, 24, 64, 85, 86, 128, 340):
        cfg, slot = _cfg(lad, io_dtype=io, batch=1, heads=heads, groups=1, head_dim=P, state_dim=N), heads * (P * N + 1) * 4
        for most in (*range(1, 1200), 1300, 2047, 2048, 2049, 4096, 8193):
            need = lad.replay_scan_workspace(cfg, most, most)
            assert need % slot == 0 and need != slot, (heads, most)


def test_sampling_needs_no_workspace(lad):
    assert {lad.replay_sample_workspace(*s) for s in ((1, 1, 1), (1, 1, 1 << 18), (256, 1, 131072), (48, 5, 50021), (1 << 20, 7, 300))} == {0}


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 64, -(1 << 32) + 64])
def test_sizes_past_32_bits_are_refused(lad, big):
    """A size that the C call's int32 would cut to another one."""
    for args in ((big, 64), (64, big)):
        with pytest.raises(lad.ReplayError, match="32 bits"):
            lad.replay_scan_workspace(_cfg(lad), *args)
    for args in ((big, 1, 8), (1, big, 8), (1, 1, big)):
        with pytest.raises(lad.ReplayError, match="32 bits"):
            lad.replay_sample_workspace(*args)
