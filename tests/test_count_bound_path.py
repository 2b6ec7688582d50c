"""Host logic: the bounds on the ring counts (csrc/count_bound.h) over appends of
as many tokens as only the device knows: whatever 0..W it takes of each
sequence (none of one whose ring they would overflow), lo <= count <= hi and
pos <= the bound on it hold, and a flush with a due sequence is not skipped."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "linear_attention_decode_amd", "csrc")
SHIM = r"""
#include "count_bound.h"
using replay::CountBound;
extern "C" {
void *cb_new(int L) { auto *b = new CountBound; b->reset(L); return b; }
void cb_free(void *h) { delete static_cast<CountBound *>(h); }
void cb_some(void *h, int W) { static_cast<CountBound *>(h)->append_some(W); }
void cb_append(void *h, int W) { static_cast<CountBound *>(h)->append(W); }
int cb_may_fold(void *h, int m) { return static_cast<CountBound *>(h)->flush_may_fold(m); }
void cb_flush(void *h, int m) { static_cast<CountBound *>(h)->flush(m); }
void cb_get(void *h, long long *out) {
    auto *b = static_cast<CountBound *>(h);
    out[0] = b->lo; out[1] = b->hi; out[2] = b->pos;
}
}
"""


@pytest.fixture(scope="module")
def cb(tmp_path_factory):
    d = tmp_path_factory.mktemp("cbp")
    src, lib = d / "shim.cpp", d / "libcbp.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.cb_new.restype = ctypes.c_void_p
    for name in ("cb_free", "cb_some", "cb_append", "cb_may_fold", "cb_flush", "cb_get"):
        getattr(L, name).argtypes = [ctypes.c_void_p] + [ctypes.c_int] * (name not in ("cb_free", "cb_get")) + [ctypes.c_void_p] * (name == "cb_get")
    return L


@pytest.mark.parametrize("L", [1, 4, 16, 32])
@pytest.mark.parametrize("seed", range(8))
def test_bounds_hold(cb, L, seed):
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 5))
    count, pos = np.zeros(B, int), np.zeros(B, int)
    h = cb.cb_new(L)
    out = (ctypes.c_longlong * 3)()
    for _ in range(200):
        what, W = r.integers(0, 3), int(r.integers(1, 2 * L + 1))
        if what == 0:
            n = r.integers(0, W + 1, B)
            n[count + n > L] = 0
            count, pos = count + n, pos + n
            cb.cb_some(h, W)
        elif what == 1:
            n = np.where(count + W <= L, W, 0)
            count, pos = count + n, pos + n
            cb.cb_append(h, W)
        else:
            due = count >= max(W, 1)
            if due.any():
                assert cb.cb_may_fold(h, W)
            count[due] = 0
            cb.cb_flush(h, W)
        cb.cb_get(h, out)
        assert out[0] <= count.min() and count.max() <= out[1] <= L and pos.max() <= out[2], (what, W)
    cb.cb_free(h)
