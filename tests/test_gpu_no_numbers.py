"""Values that are no numbers where the tests of trees and prompts do not put them: in
a tree's nodes against checkpoints of fewer bits, in the ring's entries, in a
checkpoint and in the state that a prompt goes on from."""
import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests import gpu_util as gu
from tests.test_gpu_delta import SHAPES, Prompts
from tests.test_gpu_tree import Round

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
NAMES = ["q", "k", "v", "dt", "a"]


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("read", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("which,value", [(n, NAN) for n in NAMES] + [("k", INF), ("v", INF)])
def test_in_a_node_against_a_copy(rule, io, read, which, value):
    gu.note(f"tree {value} in {which} against {read} {io} rule {rule}")
    W, at = 40, 6
    p = Round(1, 4, 2, 64, 128, 8, W, io, rule, read, seed=5, counts=[5])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    p.x[NAMES.index(which)][0, at, ..., 1] = value            # an element of every group or head, or head 1
    p.run()
    torch.cuda.synchronize()
    hit = [at] if which == "q" else [w for w in range(W) if at in ot.path(p.parent[0], w)]
    rest = [w for w in range(W) if w not in hit]
    assert torch.equal(p.y[0, rest], clean[0, rest])
    heads, cols = ([1] if which in ("dt", "a") else range(4)), ([1] if which == "v" else range(64))
    bad = torch.zeros(len(hit), 4, 64, dtype=torch.bool, device=gu.DEV)
    bad[:, [[h] for h in heads], list(cols)] = True
    y, ok = p.y[0, hit], clean[0, hit]
    assert not torch.isfinite(y[bad]).any() and torch.equal(y[~bad], ok[~bad])


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("read", [None, "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("which", NAMES[1:])
def test_in_the_ring(rule, io, read, which):
    """An entry's reaches every node, its own heads and columns alone; a slot that holds no entry reaches none."""
    gu.note(f"tree, NaN in the ring's {which} against {read} {io} rule {rule}")
    W, L, count = 20, 8, 5
    p = Round(2, 4, 2, 64, 128, L, W, io, rule, read, seed=6, counts=[count, count])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    t, base = p.layer.t, p.layer.t["base"].cpu().numpy()

    def put(b, e):
        slot = (int(base[b]) + e) % L
        if which == "k":
            t["ring_k"][b, 1, slot, 3] = NAN           # heads 2 and 3
        elif which == "v":
            t["ring_v"][b, 2, slot, 5] = NAN
        else:
            t["ring_" + which][b, slot, 2] = NAN
    for e in range(count, L):
        put(0, e)
        put(1, e)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.y, clean)
    put(0, 2)
    p.run()
    torch.cuda.synchronize()
    bad = torch.zeros(2, W, 4, 64, dtype=torch.bool, device=gu.DEV)
    bad[0, :, {"k": slice(2, 4)}.get(which, slice(2, 3)), slice(5, 6) if which == "v" else slice(None)] = True
    assert torch.equal(p.y[~bad], clean[~bad]) and not torch.isfinite(p.y[bad]).any()


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("read", [None, "bf16", "fp8"])
@pytest.mark.parametrize("P,N", [(16, 16), (64, 128)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_in_a_checkpoint(rule, io, read, P, N, value):
    """It reaches its row of the state, and so that column of every output, alone."""
    gu.note(f"tree, {value} in the checkpoint {read} P={P} N={N} {io} rule {rule}")
    p = Round(2, 4, 2, P, N, 8, 20, io, rule, read, seed=7, counts=[5, 0])
    p.run()
    torch.cuda.synchronize()
    clean = p.y.clone()
    t = p.layer.t
    if read == "fp8":
        t["s_copy"].view(torch.uint8)[0, 2, 5, 3] = 0x7F       # e4m3 has a NaN and no infinity
    else:
        t["s_master" if read is None else "s_copy"][0, 2, 5, 3] = value
    p.run()
    torch.cuda.synchronize()
    bad = torch.zeros_like(p.y, dtype=torch.bool)
    bad[0, :, 2, 5] = True
    assert torch.equal(p.y[~bad], clean[~bad]) and not torch.isfinite(p.y[bad]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("B,H", [(2, 4), (12, 16)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_in_the_state_that_a_prompt_goes_on_from(io, P, N, B, H, value):
    gu.note(f"delta_scan {value} in s_in, {B} x {H} heads P={P} N={N} {io}")
    lens = [130, 0, 64, 1, 63, 65, 10, 100, 128, 2, 70, 90][:B]
    p = Prompts(lens, H, 2, P, N, io, seed=8)
    p.run()
    torch.cuda.synchronize()
    y, S = p.y.clone(), p.s_out.clone()
    p.s_in[0, 1, 5, 3] = value
    p.s_in[1, 0, 2, 7] = value                                  # a sequence of no tokens: passed on as it is
    p.run()
    torch.cuda.synchronize()
    bad_y, bad_s = torch.zeros_like(y, dtype=torch.bool), torch.zeros_like(S, dtype=torch.bool)
    bad_y[p.rows(0), 1, 5] = True
    bad_s[0, 1, 5] = True
    bad_s[1, 0, 2, 7] = True
    assert torch.equal(p.y[~bad_y], y[~bad_y]) and not torch.isfinite(p.y[bad_y].float()).any()
    assert torch.equal(p.s_out[~bad_s], S[~bad_s]) and not torch.isfinite(p.s_out[bad_s]).any()
    assert np.array_equal(p.s_out[1, 0, 2, 7].item(), value, equal_nan=True)
