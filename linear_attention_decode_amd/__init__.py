"""Python binding of libreplayssm: the ReplaySSM decode path for Mamba-2-style
SSM layers on MI355X (gfx950).

Argument marshalling only.  Every step of the path runs in the library's HIP
kernels; torch supplies device memory and the current stream.  The entry
points keep the C names (``replay_init``, ``replay_append``, ...).
``ReplayLayer`` bundles one layer's buffers and handle for convenience.

If the built library is missing, importing this package raises ImportError:
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "ReplayError", "ReplayConfig", "ReplayBuffers", "ReplayLayer", "lib", "LIB_PATH",
    "F32", "BF16", "FP8_E4M3", "FP4_E2M1", "NONE", "SEQERR_RING_OVERFLOW", "SEQERR_ROLLBACK_RANGE",
    "SEQERR_TOO_FEW", "SEQERR_POS_OVERFLOW", "EXPORTS",
    "replay_status_string", "replay_abi_version", "replay_buffer_bytes", "replay_init",
    "replay_destroy", "replay_load_checkpoint", "replay_append", "replay_decode",
    "replay_verify", "replay_rollback", "replay_flush", "replay_step", "replay_step_layers", "replay_step_static",
    "replay_verify_step", "replay_rollback_verify_step", "replay_set_flush_skipping", "replay_get_error",
    "replay_eager_step", "replay_eager_select", "replay_stream_probe",
    "ReplayConvParams", "ReplayConv", "SEQERR_BAD_RANGE", "replay_conv_prompt", "replay_conv_step",
    "replay_scan_workspace", "replay_scan", "ReplaySampling", "replay_sample_workspace", "replay_sample",
    "replay_logprobs_workspace", "replay_logprobs", "SEQERR_BAD_TREE", "replay_delta_inputs", "replay_conv_tree",
    "replay_verify_tree", "replay_accept_tree", "replay_conv_path", "replay_append_path",
    "replay_delta_scan_workspace", "replay_delta_scan",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libreplayssm.so")

NONE, F32, BF16, FP8_E4M3, FP4_E2M1 = -1, 0, 1, 2, 3
SEQERR_RING_OVERFLOW, SEQERR_ROLLBACK_RANGE, SEQERR_TOO_FEW, SEQERR_POS_OVERFLOW = 1, 2, 4, 8
SEQERR_BAD_RANGE, SEQERR_BAD_TREE = 16, 32

# every symbol include/replayssm.h declares
EXPORTS = (
    "replay_status_string", "replay_abi_version", "replay_buffer_bytes", "replay_init",
    "replay_destroy", "replay_load_checkpoint", "replay_append", "replay_decode",
    "replay_verify", "replay_rollback", "replay_flush", "replay_step", "replay_step_layers", "replay_step_static",
    "replay_verify_step", "replay_rollback_verify_step", "replay_set_flush_skipping", "replay_get_error",
    "replay_eager_step", "replay_eager_select", "replay_stream_probe",
    "replay_conv_prompt", "replay_conv_step", "replay_scan_workspace", "replay_scan",
    "replay_sample_workspace", "replay_sample", "replay_logprobs_workspace", "replay_logprobs",
    "replay_delta_inputs", "replay_conv_tree", "replay_verify_tree", "replay_accept_tree", "replay_conv_path",
    "replay_append_path", "replay_delta_scan_workspace", "replay_delta_scan",
)

_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


class ReplayConfig(ctypes.Structure):
    _fields_ = [("batch", _I32), ("heads", _I32), ("groups", _I32), ("head_dim", _I32),
                ("state_dim", _I32), ("ring_len", _I32), ("io_dtype", _I32),
                ("read_copy", _I32), ("shared_lowp", _I32), ("rule", _I32)]


BUFFER_FIELDS = ("s_master", "s_copy", "s_scale", "ring_q", "ring_k", "ring_v", "ring_dt",
                 "ring_a", "pos", "base", "err", "sync")


class ReplayBuffers(ctypes.Structure):
    _fields_ = [(name, _VP) for name in BUFFER_FIELDS]


class ReplayConvParams(ctypes.Structure):
    _fields_ = [("width", _I32), ("slots", _I32), ("silu", _I32), ("weight", _VP), ("bias", _VP),
                ("dt_bias", _VP), ("a_log", _VP), ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class ReplaySampling(ctypes.Structure):
    _fields_ = [("temperature", _VP), ("top_k", _VP), ("top_p", _VP), ("min_p", _VP)]


class ReplayError(RuntimeError):
    pass


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "(hipcc --offload-arch=gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    L.replay_status_string.argtypes = [ctypes.c_int]
    L.replay_status_string.restype = ctypes.c_char_p
    L.replay_abi_version.restype = _I32
    L.replay_buffer_bytes.argtypes = [ctypes.POINTER(ReplayConfig), ctypes.POINTER(ctypes.c_size_t)]
    L.replay_init.argtypes = [ctypes.POINTER(ReplayConfig), ctypes.POINTER(ReplayBuffers), _VP,
                              ctypes.POINTER(_VP)]
    L.replay_destroy.argtypes = [_VP, _VP]
    L.replay_load_checkpoint.argtypes = [_VP, _VP, _VP]
    L.replay_append.argtypes = [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP]
    L.replay_decode.argtypes = [_VP, _VP, _VP]
    L.replay_verify.argtypes = [_VP, _I32, _VP, _VP]
    L.replay_rollback.argtypes = [_VP, _VP, _VP]
    L.replay_flush.argtypes = [_VP, _I32, _VP]
    L.replay_step.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP]
    L.replay_verify_step.argtypes = [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP]
    L.replay_rollback_verify_step.argtypes = [_VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP]
    L.replay_get_error.argtypes = [_VP, ctypes.POINTER(_I32), _VP, _VP]
    L.replay_set_flush_skipping.argtypes = [_VP, _I32, _VP]
    L.replay_step_static.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP]
    L.replay_step_layers.argtypes = [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP]
    L.replay_eager_step.argtypes = [ctypes.POINTER(ReplayConfig)] + [_VP] * 9
    L.replay_eager_select.argtypes = [ctypes.POINTER(ReplayConfig), _VP, _I32, _VP, _VP, _VP]
    L.replay_stream_probe.argtypes = [_I32, _VP, _VP, ctypes.c_size_t, _VP]
    L.replay_conv_prompt.argtypes = ([ctypes.POINTER(ReplayConfig), ctypes.POINTER(ReplayConvParams), _I32, _VP, _VP,
                                      _I64, _VP, _I64] + [_VP] * 10)
    L.replay_conv_step.argtypes = ([ctypes.POINTER(ReplayConfig), ctypes.POINTER(ReplayConvParams), _I32, _VP, _I64,
                                    _VP, _I64] + [_VP] * 10)
    L.replay_scan_workspace.argtypes = [ctypes.POINTER(ReplayConfig), _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]
    L.replay_scan.argtypes = ([ctypes.POINTER(ReplayConfig), _I32, _I32] + [_VP] * 11 + [ctypes.c_size_t, _VP])
    L.replay_sample_workspace.argtypes = [_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]
    L.replay_sample.argtypes = ([_I32, _I32, _I32, _VP, _I32, _I64, ctypes.POINTER(ReplaySampling)] + [_VP] * 6
                                + [ctypes.c_size_t, _VP])
    L.replay_logprobs_workspace.argtypes = [_I32, _I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]
    L.replay_logprobs.argtypes = ([_I32, _I32, _I32, _VP, _I32, _I64, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _VP,
                                   ctypes.c_size_t, _VP])
    L.replay_delta_inputs.argtypes = [ctypes.POINTER(ReplayConfig), _I32, _VP, _VP, _VP, _I64, _VP, _I64, _VP, _VP,
                                      ctypes.c_float, ctypes.c_float] + [_VP] * 5
    L.replay_delta_scan_workspace.argtypes = L.replay_scan_workspace.argtypes
    L.replay_delta_scan.argtypes = L.replay_scan.argtypes
    L.replay_conv_tree.argtypes = ([ctypes.POINTER(ReplayConfig), ctypes.POINTER(ReplayConvParams), _I32, _VP, _VP, _VP,
                                    _I64, _VP, _I64] + [_VP] * 9)
    L.replay_verify_tree.argtypes = [_VP, _I32] + [_VP] * 9
    L.replay_accept_tree.argtypes = [_I32, _I32] + [_VP] * 7
    L.replay_conv_path.argtypes = [ctypes.POINTER(ReplayConfig), ctypes.POINTER(ReplayConvParams), _I32, _VP, _VP, _VP,
                                   _I64, _VP, _VP, _VP, _VP]
    L.replay_append_path.argtypes = [_VP, _I32] + [_VP] * 8
    for name in EXPORTS:
        if name not in ("replay_status_string", "replay_abi_version"):
            getattr(L, name).restype = ctypes.c_int
    return L


lib = _load()


def _check(status: int, what: str):
    if status != 0:
        raise ReplayError(f"{what}: {lib.replay_status_string(status).decode()} (status {status})")


def _ptr(t):
    """Device pointer of a torch tensor (or None / int passthrough)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- the C entry points, same names --------------------------------------

def replay_status_string(status: int) -> str:
    return lib.replay_status_string(status).decode()


def replay_abi_version() -> int:
    return int(lib.replay_abi_version())


def replay_buffer_bytes(cfg: ReplayConfig):
    out = (ctypes.c_size_t * len(BUFFER_FIELDS))()
    _check(lib.replay_buffer_bytes(ctypes.byref(cfg), out), "replay_buffer_bytes")
    return dict(zip(BUFFER_FIELDS, [int(x) for x in out]))


def replay_init(cfg: ReplayConfig, bufs: ReplayBuffers, stream=None):
    h = _VP()
    _check(lib.replay_init(ctypes.byref(cfg), ctypes.byref(bufs), _stream(stream), ctypes.byref(h)),
           "replay_init")
    return h


def replay_destroy(h, stream=None):
    _check(lib.replay_destroy(h, _stream(stream)), "replay_destroy")


def replay_load_checkpoint(h, s_src, stream=None):
    _check(lib.replay_load_checkpoint(h, _ptr(s_src), _stream(stream)), "replay_load_checkpoint")


def replay_append(h, W, q, k, v, dt, a, stream=None):
    _check(lib.replay_append(h, W, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a), _stream(stream)),
           "replay_append")


def replay_decode(h, y, stream=None):
    _check(lib.replay_decode(h, _ptr(y), _stream(stream)), "replay_decode")


def replay_verify(h, W, y, stream=None):
    _check(lib.replay_verify(h, W, _ptr(y), _stream(stream)), "replay_verify")


def replay_rollback(h, n_reject, stream=None):
    _check(lib.replay_rollback(h, _ptr(n_reject), _stream(stream)), "replay_rollback")


def replay_flush(h, min_count, stream=None):
    _check(lib.replay_flush(h, min_count, _stream(stream)), "replay_flush")


def replay_step(h, q, k, v, dt, a, y, flush_at, stream=None):
    _check(lib.replay_step(h, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a), _ptr(y), flush_at,
                           _stream(stream)), "replay_step")


def replay_step_layers(handles, q, k, v, dt, a, y, flush_at, stream=None):
    """handles, q, k, v, dt, a, y: sequences of n entries (one per layer)."""
    n = len(handles)
    arr = lambda xs: (_VP * n)(*[_ptr(x) for x in xs])
    _check(lib.replay_step_layers((_VP * n)(*handles), n, arr(q), arr(k), arr(v), arr(dt), arr(a), arr(y),
                                  int(flush_at), _stream(stream)), "replay_step_layers")


def replay_step_static(h, q, k, v, dt, a, y, flush_at, stream=None):
    _check(lib.replay_step_static(h, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a), _ptr(y), int(flush_at),
                                  _stream(stream)), "replay_step_static")


def replay_rollback_verify_step(h, n_reject, W, q, k, v, dt, a, y, flush_at, stream=None):
    _check(lib.replay_rollback_verify_step(h, _ptr(n_reject), W, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a),
                                           _ptr(y), flush_at, _stream(stream)), "replay_rollback_verify_step")


def replay_verify_step(h, W, q, k, v, dt, a, y, flush_at, stream=None):
    _check(lib.replay_verify_step(h, W, _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(a), _ptr(y), flush_at,
                                  _stream(stream)), "replay_verify_step")


def replay_set_flush_skipping(h, enable: int, stream=None):
    _check(lib.replay_set_flush_skipping(h, int(enable), _stream(stream)), "replay_set_flush_skipping")


def replay_get_error(h, batch: int, stream=None):
    """Returns (word, per_sequence list)."""
    word = _I32()
    per = (_I32 * batch)()
    _check(lib.replay_get_error(h, ctypes.byref(word), per, _stream(stream)), "replay_get_error")
    return int(word.value), list(per)


def replay_eager_step(cfg, s_in, s_out, q, k, v, dt, a, y, stream=None):
    _check(lib.replay_eager_step(ctypes.byref(cfg), _ptr(s_in), _ptr(s_out), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(dt), _ptr(a), _ptr(y), _stream(stream)), "replay_eager_step")


def replay_eager_select(cfg, snaps, W, n_accept, s, stream=None):
    _check(lib.replay_eager_select(ctypes.byref(cfg), _ptr(snaps), W, _ptr(n_accept), _ptr(s),
                                   _stream(stream)), "replay_eager_select")


def replay_stream_probe(mode, src, dst, nbytes, stream=None):
    _check(lib.replay_stream_probe(mode, _ptr(src), _ptr(dst), nbytes, _stream(stream)),
           "replay_stream_probe")


# ---- prompts and the inputs of the recurrence -------------------------------
# These calls take torch tensors and check what their pointers cannot say:
# the kernels go by the shapes of cfg.

def _gpu():
    import torch
    return torch.cuda.current_device()


def _on(stream, gpu):
    """_stream, without building a Stream object for the current one (2.5 of a token call's 12 us on the host)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(gpu)
    return _stream(stream)


def _want(what, t, shape, dtype, gpu):
    """The address of a contiguous tensor of this shape and type on that GPU (None passes)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != gpu or not t.is_contiguous():
        raise ReplayError(f"{what}: want a contiguous {dtype} tensor of shape {shape} on the current GPU ({gpu}), got "
                          f"{t.dtype} of {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _size(what, n):
    """n, if the C call's int32 holds it (ctypes would cut it to another size)."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ReplayError(f"{what}: {n} does not fit 32 bits")
    return n


def _rows(what, t, n, width, dtype, gpu):
    """(address, row stride) of a [n, width] tensor whose rows may lie any stride apart (None: (None, 0))."""
    if t is None:
        return None, 0
    if t.shape != (n, width) or t.dtype is not dtype or t.get_device() != gpu or (width > 1 and t.stride(1) != 1):
        raise ReplayError(f"{what}: want a {dtype} tensor of shape {(n, width)} with unit stride along its rows on the "
                          f"current GPU ({gpu}), got {t.dtype} of {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr(), (t.stride(0) if n > 1 else max(t.stride(0), width))


def _io_type(cfg):
    import torch
    return torch.bfloat16 if cfg.io_dtype == BF16 else torch.float32


class ReplayConv:
    """The convolution and discretisation of one layer (replay_conv_params):
    weight [C, K] and bias [C] f32, dt_bias and a_log [H] f32 (None where the
    layer has none), `slots` rows of state a sequence (K - 1 + W serves
    rounds of W drafts).  Holds its tensors."""

    def __init__(self, weight, bias=None, dt_bias=None, a_log=None, slots=None, silu=True, dt_min=0.0,
                 dt_max=float("inf")):
        import torch
        channels, self.width = weight.shape
        self.channels, self.slots = channels, self.width - 1 if slots is None else int(slots)
        heads = next((t.shape for t in (a_log, dt_bias) if t is not None), None)
        self.heads = None if heads is None else heads[0]
        self.tensors = (weight, bias, dt_bias, a_log)
        f32, gpu = torch.float32, _gpu()
        self.gpu = gpu
        self.params = ReplayConvParams(
            self.width, self.slots, int(bool(silu)), _want("weight", weight, (channels, self.width), f32, gpu),
            _want("bias", bias, (channels,), f32, gpu), _want("dt_bias", dt_bias, (self.heads,), f32, gpu),
            _want("a_log", a_log, (self.heads,), f32, gpu), dt_min, 0.0 if dt_max == float("inf") else dt_max)


def _conv_call(what, cfg, conv, n, lead, x, dt_raw, q, k, v, dt, a, io, f32, gpu):
    """What the two convolution calls share: x, its stride, dt_raw, its stride; and q, k, v, dt, a."""
    H, G, P, N = cfg.heads, cfg.groups, cfg.head_dim, cfg.state_dim
    C = H * P + 2 * G * N
    if conv.channels != C or (dt_raw is not None and conv.heads != H):
        raise ReplayError(f"{what}: a convolution of {conv.channels} channels and {conv.heads} heads for a layer of "
                          f"{C} channels and {H} heads")
    if conv.gpu != gpu:
        raise ReplayError(f"{what}: the convolution's tensors are on GPU {conv.gpu}, the current one is {gpu}")
    rows = _rows("x", x, n, C, io, gpu) + _rows("dt_raw", dt_raw, n, H, io, gpu)
    outs = (_want("q", q, (*lead, G, N), io, gpu), _want("k", k, (*lead, G, N), io, gpu),
            _want("v", v, (*lead, H, P), io, gpu))
    if dt_raw is None:
        return rows, (*outs, None, None)
    return rows, (*outs, _want("dt", dt, (*lead, H), f32, gpu), _want("a", a, (*lead, H), f32, gpu))


def replay_conv_prompt(cfg, conv, T, cu_seqlens, x, dt_raw, pos, state_in, state_out, q, k, v, dt, a, err, stream=None):
    """x [T, C] and dt_raw [T, H] may be views into wider rows; conv: ReplayConv; pos, state_in, dt_raw may be None."""
    import torch
    i32, io, gpu, B = torch.int32, _io_type(cfg), _gpu(), cfg.batch
    rows, outs = _conv_call("replay_conv_prompt", cfg, conv, T, (T,), x, dt_raw, q, k, v, dt, a, io, torch.float32, gpu)
    state = (B, conv.slots, conv.channels)
    _check(lib.replay_conv_prompt(
        ctypes.byref(cfg), ctypes.byref(conv.params), T, _want("cu_seqlens", cu_seqlens, (B + 1,), i32, gpu), *rows,
        _want("pos", pos, (B,), i32, gpu), _want("state_in", state_in, state, io, gpu),
        _want("state_out", state_out, state, io, gpu), *outs, _want("err", err, (B + 1,), i32, gpu), _on(stream, gpu)),
        "replay_conv_prompt")


def replay_conv_step(cfg, conv, W, x, dt_raw, pos, conv_state, q, k, v, dt, a, base=None, n_reject=None, stream=None):
    """x [B W, C] and dt_raw [B W, H] may be views into wider rows; conv: ReplayConv; dt_raw may be None."""
    import torch
    i32, io, gpu, B = torch.int32, _io_type(cfg), _gpu(), cfg.batch
    rows, outs = _conv_call("replay_conv_step", cfg, conv, B * W, (B, W), x, dt_raw, q, k, v, dt, a, io, torch.float32,
                            gpu)
    _check(lib.replay_conv_step(
        ctypes.byref(cfg), ctypes.byref(conv.params), W, *rows, _want("pos", pos, (B,), i32, gpu),
        _want("base", base, (B,), i32, gpu), _want("n_reject", n_reject, (B,), i32, gpu),
        _want("conv_state", conv_state, (B, conv.slots, conv.channels), io, gpu), *outs, _on(stream, gpu)),
        "replay_conv_step")


def _scan_workspace(what, cfg, T, max_len) -> int:
    n = ctypes.c_size_t()
    _check(getattr(lib, what)(ctypes.byref(cfg), _size("T", T), _size("max_len", max_len), ctypes.byref(n)), what)
    return n.value


def replay_scan_workspace(cfg, T, max_len) -> int:
    """Bytes of workspace that replay_scan needs for T rows, up to max_len of them a sequence."""
    return _scan_workspace("replay_scan_workspace", cfg, T, max_len)


def _workspace(t, gpu):
    """(address, bytes) of a contiguous tensor of any type (None: (None, 0))."""
    if t is None:
        return None, 0
    if t.get_device() != gpu or not t.is_contiguous():
        raise ReplayError(f"workspace: want a contiguous tensor on the current GPU ({gpu}), got one on {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _scan(what, cfg, T, max_len, cu_seqlens, q, k, v, dt, a, s_in, s_out, y, err, workspace, stream, names):
    import torch
    f32, i32, io, gpu = torch.float32, torch.int32, _io_type(cfg), _gpu()
    B, H, G, P, N = cfg.batch, cfg.heads, cfg.groups, cfg.head_dim, cfg.state_dim
    _check(getattr(lib, what)(
        ctypes.byref(cfg), _size("T", T), _size("max_len", max_len), _want("cu_seqlens", cu_seqlens, (B + 1,), i32, gpu),
        _want("q", q, (T, G, N), io, gpu), _want("k", k, (T, G, N), io, gpu), _want("v", v, (T, H, P), io, gpu),
        _want(names[0], dt, (T, H), f32, gpu), _want(names[1], a, (T, H), f32, gpu),
        _want("s_in", s_in, (B, H, P, N), f32, gpu), _want("s_out", s_out, (B, H, P, N), f32, gpu),
        _want("y", y, (T, H, P), io, gpu), _want("err", err, (B + 1,), i32, gpu), *_workspace(workspace, gpu),
        _on(stream, gpu)), what)


def replay_scan(cfg, T, max_len, cu_seqlens, q, k, v, dt, a, s_in, s_out, y, err, workspace=None, stream=None):
    """Packed prompts: q, k [T, G, N], v and y [T, H, P], dt, a [T, H]; s_in may be None (zeros)."""
    _scan("replay_scan", cfg, T, max_len, cu_seqlens, q, k, v, dt, a, s_in, s_out, y, err, workspace, stream, ("dt", "a"))


def replay_sample_workspace(B, W, V) -> int:
    """Bytes of workspace that replay_sample needs for B sequences of W positions and V logits: always 0."""
    n = ctypes.c_size_t()
    _check(lib.replay_sample_workspace(_size("B", B), _size("W", W), _size("V", V), ctypes.byref(n)),
           "replay_sample_workspace")
    return n.value


def _logit_rows(logits, gpu):
    """The row stride of logits [B, W, V]."""
    import torch
    B, W, V = logits.shape
    row = logits.stride(1) if W > 1 else logits.stride(0) if B > 1 else V
    if (logits.dtype not in (torch.float32, torch.bfloat16) or logits.get_device() != gpu
            or (V > 1 and logits.stride(2) != 1) or (B > 1 and logits.stride(0) != W * row)):
        raise ReplayError("logits: want a float32 or bf16 tensor [B, W, V] of evenly spaced rows with unit stride along "
                          f"them on the current GPU ({gpu}), got {logits.dtype} with strides {logits.stride()} on "
                          f"{logits.device}")
    return row


def replay_sample(logits, u, tokens, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, fed=None,
                  n_reject=None, workspace=None, stream=None):
    """logits [B, W, V] (float32 or bf16; positions may lie any stride apart), u [B, W] f32, tokens [B, W] int32;
    temperature, top_p, min_p [B] f32 and top_k [B] int32 (None: off); probs [B, W] f32; fed [B, W] and n_reject [B]
    int32 for the rounds of drafts."""
    import torch
    f32, i32, gpu = torch.float32, torch.int32, _gpu()
    B, W, V = logits.shape
    row = _logit_rows(logits, gpu)
    opt = ReplaySampling(_want("temperature", temperature, (B,), f32, gpu), _want("top_k", top_k, (B,), i32, gpu),
                         _want("top_p", top_p, (B,), f32, gpu), _want("min_p", min_p, (B,), f32, gpu))
    _check(lib.replay_sample(
        B, W, V, logits.data_ptr(), F32 if logits.dtype is f32 else BF16, row, ctypes.byref(opt),
        _want("u", u, (B, W), f32, gpu), _want("tokens", tokens, (B, W), i32, gpu), _want("probs", probs, (B, W), f32, gpu),
        _want("fed", fed, (B, W), i32, gpu), _want("n_reject", n_reject, (B,), i32, gpu), *_workspace(workspace, gpu),
        _on(stream, gpu)), "replay_sample")


def replay_logprobs_workspace(B, W, V, n_top) -> int:
    """Bytes of workspace that replay_logprobs needs for B sequences of W positions, V logits and n_top alternatives."""
    n = ctypes.c_size_t()
    _check(lib.replay_logprobs_workspace(_size("B", B), _size("W", W), _size("V", V), _size("n_top", n_top), ctypes.byref(n)),
           "replay_logprobs_workspace")
    return n.value


def replay_logprobs(logits, ids=None, logp=None, entropy=None, top_ids=None, top_logp=None, temperature=None,
                    workspace=None, stream=None):
    """logits [B, W, V] as for replay_sample; ids [B, W, M] int32 with logp [B, W, M] f32; entropy [B, W] f32; top_ids
    [B, W, n] int32 with top_logp [B, W, n] f32; temperature [B] f32 (None: 1).  Any of the outputs may be None."""
    import torch
    f32, i32, gpu = torch.float32, torch.int32, _gpu()
    B, W, V = logits.shape
    row = _logit_rows(logits, gpu)
    for what, a, b in (("ids and logp", ids, logp), ("top_ids and top_logp", top_ids, top_logp)):
        if (a is None) != (b is None) or (a is not None and a.dim() != 3):
            raise ReplayError(f"{what}: want both, of shape (B, W, count), or neither")
    M, n = (0 if t is None else t.shape[2] for t in (ids, top_ids))
    _check(lib.replay_logprobs(
        B, W, V, logits.data_ptr(), F32 if logits.dtype is f32 else BF16, row, _want("temperature", temperature, (B,), f32, gpu),
        M, _want("ids", ids, (B, W, M), i32, gpu), _want("logp", logp, (B, W, M), f32, gpu),
        _want("entropy", entropy, (B, W), f32, gpu), n, _want("top_ids", top_ids, (B, W, n), i32, gpu),
        _want("top_logp", top_logp, (B, W, n), f32, gpu), *_workspace(workspace, gpu), _on(stream, gpu)), "replay_logprobs")


# ---- Gated DeltaNet layers' inputs; trees of drafted tokens -------------------

def replay_delta_inputs(cfg, T, q_in, k_in, b_raw, a_raw, dt_bias, a_log, q_scale, eps, q, k, beta, alpha, stream=None):
    """T rows: q_in, k_in, q, k [T, G, N] (q may be q_in, k k_in); b_raw, a_raw [T, H] may be views into wider rows;
    dt_bias (or None) and a_log [H] f32; beta, alpha [T, H] f32."""
    import torch
    f32, io, gpu = torch.float32, _io_type(cfg), _gpu()
    H, qk = cfg.heads, (T, cfg.groups, cfg.state_dim)
    _check(lib.replay_delta_inputs(
        ctypes.byref(cfg), _size("T", T), _want("q_in", q_in, qk, io, gpu), _want("k_in", k_in, qk, io, gpu),
        *_rows("b_raw", b_raw, T, H, io, gpu), *_rows("a_raw", a_raw, T, H, io, gpu), _want("dt_bias", dt_bias, (H,), f32, gpu),
        _want("a_log", a_log, (H,), f32, gpu), q_scale, eps, _want("q", q, qk, io, gpu), _want("k", k, qk, io, gpu),
        _want("beta", beta, (T, H), f32, gpu), _want("alpha", alpha, (T, H), f32, gpu), _on(stream, gpu)),
        "replay_delta_inputs")


def replay_delta_scan_workspace(cfg, T, max_len) -> int:
    """Bytes of workspace that replay_delta_scan needs for T rows, up to max_len of them a sequence."""
    return _scan_workspace("replay_delta_scan_workspace", cfg, T, max_len)


def replay_delta_scan(cfg, T, max_len, cu_seqlens, q, k, v, beta, alpha, s_in, s_out, y, err, workspace=None, stream=None):
    """Packed prompts of a Gated DeltaNet layer: q, k [T, G, N], v and y [T, H, P], beta, alpha [T, H]; s_in may be None."""
    _scan("replay_delta_scan", cfg, T, max_len, cu_seqlens, q, k, v, beta, alpha, s_in, s_out, y, err, workspace, stream,
          ("beta", "alpha"))


def _tree(parent, n_nodes, B, W, gpu):
    import torch
    return _want("parent", parent, (B, W), torch.int32, gpu), _want("n_nodes", n_nodes, (B,), torch.int32, gpu)


def _path(path, n_keep, B, W, gpu):
    import torch
    return _want("path", path, (B, W), torch.int32, gpu), _want("n_keep", n_keep, (B,), torch.int32, gpu)


def _nodes(cfg, W, q, k, v, dt, a, gpu):
    import torch
    f32, io, B, H = torch.float32, _io_type(cfg), cfg.batch, cfg.heads
    qk = (B, W, cfg.groups, cfg.state_dim)
    return (_want("q", q, qk, io, gpu), _want("k", k, qk, io, gpu), _want("v", v, (B, W, H, cfg.head_dim), io, gpu),
            _want("dt", dt, (B, W, H), f32, gpu), _want("a", a, (B, W, H), f32, gpu))


def replay_conv_tree(cfg, conv, W, parent, x, dt_raw, pos, conv_state, q, k, v, dt, a, err, n_nodes=None, stream=None):
    """parent [B, W] int32, n_nodes [B] int32 (None: W each); x [B W, C] and dt_raw [B W, H] may be views into wider rows;
    conv: ReplayConv; dt_raw may be None."""
    import torch
    i32, io, gpu, B = torch.int32, _io_type(cfg), _gpu(), cfg.batch
    rows, outs = _conv_call("replay_conv_tree", cfg, conv, B * W, (B, W), x, dt_raw, q, k, v, dt, a, io, torch.float32,
                            gpu)
    _check(lib.replay_conv_tree(
        ctypes.byref(cfg), ctypes.byref(conv.params), W, *_tree(parent, n_nodes, B, W, gpu), *rows,
        _want("pos", pos, (B,), i32, gpu), _want("conv_state", conv_state, (B, conv.slots, conv.channels), io, gpu), *outs,
        _want("err", err, (B + 1,), i32, gpu), _on(stream, gpu)), "replay_conv_tree")


def replay_conv_path(cfg, conv, W, path, n_keep, x, pos, conv_state, err, stream=None):
    """path [B, W] and n_keep [B] as replay_accept_tree gives them; x as for replay_conv_tree."""
    import torch
    i32, io, gpu, B = torch.int32, _io_type(cfg), _gpu(), cfg.batch
    C = cfg.heads * cfg.head_dim + 2 * cfg.groups * cfg.state_dim
    if conv.channels != C or conv.gpu != gpu:
        raise ReplayError(f"replay_conv_path: a convolution of {conv.channels} channels on GPU {conv.gpu} for a layer of {C} "
                          f"on the current one, {gpu}")
    _check(lib.replay_conv_path(
        ctypes.byref(cfg), ctypes.byref(conv.params), W, *_path(path, n_keep, B, W, gpu), *_rows("x", x, B * W, C, io, gpu),
        _want("pos", pos, (B,), i32, gpu), _want("conv_state", conv_state, (B, conv.slots, C), io, gpu),
        _want("err", err, (B + 1,), i32, gpu), _on(stream, gpu)), "replay_conv_path")


def replay_accept_tree(parent, tokens, fed, path, n_keep, n_nodes=None, stream=None):
    """parent, tokens, fed, path [B, W] and n_keep, n_nodes [B], all int32 (n_nodes None: W each)."""
    import torch
    i32, gpu = torch.int32, _gpu()
    B, W = parent.shape
    up, n = _tree(parent, n_nodes, B, W, gpu)
    _check(lib.replay_accept_tree(B, W, up, n, _want("tokens", tokens, (B, W), i32, gpu), _want("fed", fed, (B, W), i32, gpu),
                                  *_path(path, n_keep, B, W, gpu), _on(stream, gpu)), "replay_accept_tree")


# The handle does not tell its shapes: cfg is its layer's.

def replay_verify_tree(h, cfg, W, parent, q, k, v, dt, a, y, n_nodes=None, stream=None):
    """q, k [B, W, G, N], v [B, W, H, P], dt, a [B, W, H], y [B, W, H, P] f32; cfg: the layer's, its shapes are checked."""
    import torch
    gpu = _gpu()
    _check(lib.replay_verify_tree(h, W, *_tree(parent, n_nodes, cfg.batch, W, gpu), *_nodes(cfg, W, q, k, v, dt, a, gpu),
                                  _want("y", y, (cfg.batch, W, cfg.heads, cfg.head_dim), torch.float32, gpu),
                                  _on(stream, gpu)), "replay_verify_tree")


def replay_append_path(h, cfg, W, path, n_keep, q, k, v, dt, a, stream=None):
    """Nodes path[b, :n_keep[b]] of replay_verify_tree's arguments into the ring; cfg: the layer's, its shapes are checked."""
    gpu = _gpu()
    _check(lib.replay_append_path(h, W, *_path(path, n_keep, cfg.batch, W, gpu), *_nodes(cfg, W, q, k, v, dt, a, gpu),
                                  _on(stream, gpu)), "replay_append_path")


# ---- one layer's state, allocated with torch -------------------------------

_DTYPE_CODE = {"f32": F32, "bf16": BF16, "fp8": FP8_E4M3, "fp4": FP4_E2M1, None: NONE, "none": NONE}
# replay_rule: the layer's recurrence ("mamba2": S = a S + dt v k^T; "gdn": the
# gated delta rule, dt carrying beta and a carrying alpha)
RULE_CODE = {"mamba2": 0, "gdn": 1}
MAMBA2, GATED_DELTA = 0, 1


class ReplayLayer:
    """Buffers + handle of one SSM layer's decode state on the current GPU.

    Tensors (torch, on `device`): s_master [B,H,P,N] f32 (absent in shared
    mode), s_copy [B,H,P,N] bf16/uint8 or [B,H,P*N/2] uint8 FP4 codes (when
    read_copy is set), s_scale [B,H] f32 (e4m3) or [B,H,P*N/32] uint8 E8M0
    (FP4), ring_q/ring_k [B,G,L,N], ring_v [B,H,L,P] (io
    dtype), ring_dt/ring_a [B,L,H] f32 (slot-major), pos/base [B] int32, err [B+1] int32,
    sync [B, G+1, 32] int32 (arrival counters, one per 128-byte line; not
    allocated with counters=False, for a layer stepped by step_static only).
    """

    def __init__(self, batch, heads, groups, head_dim, state_dim, ring_len, io_dtype="bf16",
                 read_copy=None, shared_lowp=False, device="cuda", stream=None, counters=True, rule="mamba2"):
        import torch
        self.cfg = ReplayConfig(batch, heads, groups, head_dim, state_dim, ring_len,
                                _DTYPE_CODE[io_dtype], _DTYPE_CODE[read_copy], int(bool(shared_lowp)),
                                RULE_CODE[rule])
        self.rule = rule
        self.io_dtype = io_dtype
        self.read_copy = read_copy
        nbytes = replay_buffer_bytes(self.cfg)
        B, H, G, P, N, L = batch, heads, groups, head_dim, state_dim, ring_len
        iot = torch.bfloat16 if io_dtype == "bf16" else torch.float32
        copy_t = torch.bfloat16 if read_copy == "bf16" else torch.uint8
        fp4 = read_copy == "fp4"
        shapes = {
            "s_master": ((B, H, P, N), torch.float32),
            "s_copy": ((B, H, P * N // 2) if fp4 else (B, H, P, N), copy_t),
            "s_scale": ((B, H, P * N // 32), torch.uint8) if fp4 else ((B, H), torch.float32),
            "ring_q": ((B, G, L, N), iot),
            "ring_k": ((B, G, L, N), iot), "ring_v": ((B, H, L, P), iot),
            "ring_dt": ((B, L, H), torch.float32), "ring_a": ((B, L, H), torch.float32),
            "pos": ((B,), torch.int32), "base": ((B,), torch.int32), "err": ((B + 1,), torch.int32),
            "sync": ((B, G + 1, 32), torch.int32),
        }
        self.t = {}
        for name in BUFFER_FIELDS:
            if nbytes[name] == 0 or (name == "sync" and not counters):
                self.t[name] = None
                continue
            shape, dt = shapes[name]
            t = torch.empty(shape, dtype=dt, device=device)
            assert t.numel() * t.element_size() == nbytes[name], name
            self.t[name] = t
        self.bufs = ReplayBuffers(*[_ptr(self.t[n]) for n in BUFFER_FIELDS])
        self.h = replay_init(self.cfg, self.bufs, stream)

    def __getattr__(self, name):
        t = self.__dict__.get("t")
        if t is not None and name in t:
            return t[name]
        raise AttributeError(name)

    def append(self, W, q, k, v, dt, a, stream=None):
        replay_append(self.h, W, q, k, v, dt, a, stream)

    def decode(self, y, stream=None):
        replay_decode(self.h, y, stream)

    def verify(self, W, y, stream=None):
        replay_verify(self.h, W, y, stream)

    def rollback(self, n_reject, stream=None):
        replay_rollback(self.h, n_reject, stream)

    def flush(self, min_count, stream=None):
        replay_flush(self.h, min_count, stream)

    def step(self, q, k, v, dt, a, y, flush_at=None, stream=None):
        replay_step(self.h, q, k, v, dt, a, y, self.cfg.ring_len if flush_at is None else flush_at, stream)

    def step_static(self, q, k, v, dt, a, y, flush_at=None, stream=None):
        """replay_step with the library's static arrival counters (no `sync` buffer needed)."""
        replay_step_static(self.h, q, k, v, dt, a, y, self.cfg.ring_len if flush_at is None else flush_at, stream)

    def verify_step(self, W, q, k, v, dt, a, y, flush_at=None, stream=None):
        """Fold if due (count >= flush_at, default L - W + 1), append W drafts, score them."""
        fa = self.cfg.ring_len - W + 1 if flush_at is None else flush_at
        replay_verify_step(self.h, W, q, k, v, dt, a, y, fa, stream)

    def rollback_verify_step(self, n_reject, W, q, k, v, dt, a, y, flush_at=None, stream=None):
        """rollback(n_reject), then verify_step(W, ...), fused where the round is one launch."""
        fa = self.cfg.ring_len - W + 1 if flush_at is None else flush_at
        replay_rollback_verify_step(self.h, n_reject, W, q, k, v, dt, a, y, fa, stream)

    def conv_prompt(self, conv, T, cu_seqlens, x, dt_raw, state_in, state_out, q, k, v, dt, a, stream=None):
        """The inputs of packed prompts (replay_conv_prompt), their last rows kept for this layer's next tokens."""
        replay_conv_prompt(self.cfg, conv, T, cu_seqlens, x, dt_raw, self.t["pos"], state_in, state_out, q, k, v, dt, a,
                           self.t["err"], stream)

    def conv_step(self, conv, W, x, dt_raw, conv_state, q, k, v, dt, a, n_reject=None, stream=None):
        """The inputs of the next W tokens; n_reject: the rollback that the coming rollback_verify_step applies."""
        replay_conv_step(self.cfg, conv, W, x, dt_raw, self.t["pos"], conv_state, q, k, v, dt, a, self.t["base"],
                         n_reject, stream)

    def scan(self, T, max_len, cu_seqlens, q, k, v, dt, a, s_in, s_out, y, workspace=None, stream=None):
        """The recurrence over packed prompts (replay_scan, or replay_delta_scan: dt is beta, a alpha);
        load_checkpoint(s_out) makes its states this layer's."""
        scan = replay_delta_scan if self.cfg.rule == GATED_DELTA else replay_scan
        scan(self.cfg, T, max_len, cu_seqlens, q, k, v, dt, a, s_in, s_out, y, self.t["err"], workspace, stream)

    def conv_tree(self, conv, W, parent, x, dt_raw, conv_state, q, k, v, dt, a, n_nodes=None, stream=None):
        """The inputs of a tree of drafts (replay_conv_tree)."""
        replay_conv_tree(self.cfg, conv, W, parent, x, dt_raw, self.t["pos"], conv_state, q, k, v, dt, a, self.t["err"], n_nodes,
                         stream)

    def verify_tree(self, W, parent, q, k, v, dt, a, y, n_nodes=None, stream=None):
        """Outputs of a tree of drafts; the ring and the pointers stay as they are."""
        replay_verify_tree(self.h, self.cfg, W, parent, q, k, v, dt, a, y, n_nodes, stream)

    def conv_path(self, conv, W, path, n_keep, x, conv_state, stream=None):
        """The kept path's rows into the convolution's state, ahead of append_path."""
        replay_conv_path(self.cfg, conv, W, path, n_keep, x, self.t["pos"], conv_state, self.t["err"], stream)

    def append_path(self, W, path, n_keep, q, k, v, dt, a, stream=None):
        """The kept path of a tree into the ring."""
        replay_append_path(self.h, self.cfg, W, path, n_keep, q, k, v, dt, a, stream)

    def load_checkpoint(self, s_src, stream=None):
        replay_load_checkpoint(self.h, s_src, stream)

    def set_flush_skipping(self, enable: bool, stream=None):
        replay_set_flush_skipping(self.h, 1 if enable else 0, stream)

    def get_error(self, stream=None):
        return replay_get_error(self.h, self.cfg.batch, stream)

    def close(self, stream=None):
        if self.h is not None:
            replay_destroy(self.h, stream)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
