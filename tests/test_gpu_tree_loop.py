"""The prompt, tree, sampling and log-probability calls together, as a serving
loop uses them: prompts through the convolution (and a Gated DeltaNet layer's
inputs) and the scan into the layer, then rounds of trees -- the nodes'
convolution, their outputs, tokens behind them with their log-probabilities,
the path that these confirm, its rows into the convolution's state and the
ring, a flush -- with nothing of the loop on the host but its launches: on the
current stream, on another one, or as two captured graphs that are replayed
with the next round's drafts.

Afterwards, for the tokens that were accepted: v (and for Mamba-2 q and k) to
the convolution's float64 form, within its own bound, 1.1 (K + 1) 2^-24 of its
magnitudes and the activation's and the io type's rounding; a Gated DeltaNet
layer's q and k to unit rows of that form (a row's relative error twice over)
and its gates to theirs; the outputs to the float64 recurrence over the layer's
own inputs, within (3 n + 2 N + 128) 2^-24 of their magnitudes for n tokens, eight
times as much for the gated delta rule (as its scan's and its trees' bounds are),
and for bf16 io 2^-15 more (the prompt's products), the prompt's outputs one
rounding more; the log-probabilities to the logits', 2^-18 absolute: 61 terms
of magnitude 1, an exponential and a logarithm."""
import contextlib

import numpy as np
import pytest
import torch

from oracle import prompt as op
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
PARENT = [-1, 0, 0, 1, 1, 2, 3]
CHILD = [0, 0, 1, 0, 1, 0, 0]     # which of its parent's drafts a node is


@pytest.mark.parametrize("mode", ["current", "stream", "graph"])
@pytest.mark.parametrize("rule,io,lens,H,G,P,N,K", [
    (0, "f32", [9, 1, 40], 4, 2, 64, 128, 4), (0, "bf16", [70, 33], 6, 2, 64, 64, 3),
    (1, "f32", [33, 1, 64, 20], 4, 2, 64, 64, 4), (1, "bf16", [150, 37], 6, 3, 128, 128, 4)])
def test_prompts_then_rounds_of_trees(mode, rule, io, lens, H, G, P, N, K):
    import linear_attention_decode_amd as lad
    gu.note(f"tree loop {mode} rule={rule} {io} {lens}")
    B, V, W, L, rounds = len(lens), 61, len(PARENT), 16, 10
    r = np.random.default_rng(sum(lens) + rule)
    t_io = torch.bfloat16 if io == "bf16" else torch.float32
    C, f32, i32, raws = H * P + 2 * G * N, torch.float32, torch.int32, (2 if rule else 1) * H
    dev = lambda a, t=f32: torch.from_numpy(np.array(a)).to(t).to(gu.DEV)  # noqa: E731
    table = dev(r.standard_normal((V, C + raws)), t_io)
    back = dev(r.standard_normal((H * P, V)) / np.sqrt(H * P))
    weight, bias = r.uniform(-0.6, 0.6, (C, K)).astype(np.float32), r.uniform(-0.3, 0.3, C).astype(np.float32)
    dt_bias, a_log = r.uniform(-4, -1, H).astype(np.float32), np.log(r.uniform(1, 8, H)).astype(np.float32)
    conv = lad.ReplayConv(dev(weight), dev(bias), dev(dt_bias), dev(a_log), slots=K - 1 + W)
    layer = lad.ReplayLayer(B, H, G, P, N, L, io_dtype=io, rule="gdn" if rule else "mamba2", device=gu.DEV)
    guess = lambda t, c: (t * 7 + 5 + 11 * c) % V   # noqa: E731  what follows a token, in the drafts' opinion
    parent = dev(np.tile(PARENT, (B, 1)), i32)
    side = torch.cuda.Stream() if mode == "stream" else None
    on = (lambda: torch.cuda.stream(side)) if side else contextlib.nullcontext
    at = (lambda: dict(stream=side)) if side else dict

    def gates(n, x, q, k, dt, a):
        if rule:
            lad.replay_delta_inputs(layer.cfg, n, q.view(n, G, N), k.view(n, G, N), x[:, C:C + H], x[:, C + H:], conv.tensors[2],
                                    conv.tensors[3], N ** -0.5, 1e-6, q.view(n, G, N), k.view(n, G, N), dt.view(n, H), a.view(n, H), **at())

    def logits(y, fed):   # the drafts are often right, the first one more so
        out = (y.float().reshape(-1, H * P) @ back).reshape(*fed.shape, V)
        for c, lure in ((0, 3.0), (1, 2.5)):
            out = out.scatter_add(-1, guess(fed, c).long().unsqueeze(-1), torch.full((*fed.shape, 1), lure, device=gu.DEV))
        return out.contiguous()

    mk = lambda *s: (*(torch.empty(*s, G, N, dtype=t_io, device=gu.DEV) for _ in range(2)),   # noqa: E731
                     torch.empty(*s, H, P, dtype=t_io, device=gu.DEV), *(torch.empty(*s, H, device=gu.DEV) for _ in range(2)))
    prompts, ends, T = [r.integers(0, V, n) for n in lens], np.cumsum(lens), sum(lens)
    cu, state = dev([0, *ends], i32), torch.full((B, conv.slots, C), float("nan"), dtype=t_io, device=gu.DEV)
    px, pin = table[dev(np.concatenate(prompts), torch.long)], mk(T)
    py, S = torch.empty(T, H, P, dtype=t_io, device=gu.DEV), torch.empty(B, H, P, N, device=gu.DEV)
    u = dev(r.uniform(0, 1, (rounds + 1, B, W)))
    settings = dict(temperature=dev([0.8] * B), top_k=dev([20] * B, i32), top_p=dev([0.95] * B), min_p=dev([0.01] * B))
    need = (lad.replay_delta_scan_workspace if rule else lad.replay_scan_workspace)(layer.cfg, T, max(lens))
    workspace = torch.empty(need, dtype=torch.uint8, device=gu.DEV) if need else None
    token = torch.empty(B, 1, dtype=i32, device=gu.DEV)
    x, fed = torch.empty(B * W, C + raws, dtype=t_io, device=gu.DEV), torch.empty(B, W, dtype=i32, device=gu.DEV)
    ins, y, lg, uu = mk(B, W), torch.empty(B, W, H, P, device=gu.DEV), torch.empty(B, W, V, device=gu.DEV), torch.empty(B, W, device=gu.DEV)
    tokens, path, keep = (torch.empty(*s, dtype=i32, device=gu.DEV) for s in ((B, W), (B, W), (B,)))
    logp, lws = torch.empty(B, W, device=gu.DEV), lad.replay_logprobs_workspace(B, W, V, 0)
    lws = torch.empty(lws, dtype=torch.uint8, device=gu.DEV) if lws else None
    torch.cuda.synchronize()

    def nodes():
        layer.conv_tree(conv, W, parent, x[:, :C], None if rule else x[:, C:], state, ins[0], ins[1], ins[2],
                        *((None, None) if rule else ins[3:]), **at())
        gates(B * W, x, ins[0], ins[1], ins[3], ins[4])
        layer.verify_tree(W, parent, *ins, y, **at())

    def confirm():
        lad.replay_sample(lg, uu, tokens, **settings, **at())
        lad.replay_logprobs(lg, tokens.view(B, W, 1), logp.view(B, W, 1), workspace=lws, **at())
        lad.replay_accept_tree(parent, tokens, fed, path, keep, **at())
        layer.conv_path(conv, W, path, keep, x[:, :C], state, **at())
        layer.append_path(W, path, keep, *ins, **at())
        layer.flush(L - W + 1, **at())

    with on():
        layer.conv_prompt(conv, T, cu, px[:, :C], None if rule else px[:, C:], None, state, *pin[:3],
                          *((None, None) if rule else pin[3:]), **at())
        gates(T, px, pin[0], pin[1], pin[3], pin[4])
        layer.scan(T, max(lens), cu, *pin, None, S, py, workspace, **at())
        layer.load_checkpoint(S, **at())
        last = dev([p[-1] for p in prompts], i32).unsqueeze(1)
        lad.replay_sample(logits(py[dev(ends - 1, torch.long)], last), u[rounds, :, :1].contiguous(), token, **settings, **at())
        graphs = None
        if mode == "graph":
            torch.cuda.synchronize()
            graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
            for g, f in zip(graphs, (nodes, confirm)):
                with torch.cuda.graph(g):
                    f()
        kept = []
        for rd in range(rounds):
            cols = [token]
            for w in range(1, W):
                cols.append(guess(cols[PARENT[w]], CHILD[w]))
            fed.copy_(torch.cat(cols, 1))
            x.copy_(table[fed.reshape(-1).long()])
            uu.copy_(u[rd])
            graphs[0].replay() if graphs else nodes()
            lg.copy_(logits(y, fed))
            graphs[1].replay() if graphs else confirm()
            token = tokens.gather(1, path.gather(1, (keep - 1).long().unsqueeze(1)).long())
            kept.append([t.clone() for t in (fed, path, keep, tokens, y, lg, logp, *ins)])
    torch.cuda.synchronize()
    assert layer.get_error()[0] == 0

    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    eps, accepted = 2.0 ** -8 if io == "bf16" else E24, 0
    kept = [[host(t) for t in rd] for rd in kept]
    for b, n in enumerate(lens):
        steps = []   # of each round its accepted nodes
        for fd, pth, kp, tok, *_ in kept:
            nodes_ = pth[b, :int(kp[b])].astype(int)
            assert nodes_[0] == 0 and np.all(pth[b, len(nodes_):] == -1)
            for p, c in zip(nodes_, nodes_[1:]):
                assert PARENT[c] == p and fd[b, c] == tok[b, p]
            children = [w for w in range(W) if PARENT[w] == nodes_[-1]]
            assert all(fd[b, w] != tok[b, nodes_[-1]] for w in children)   # it goes no further
            steps.append(nodes_)
        accepted += sum(map(len, steps))
        for rd, p in zip(kept, steps):
            z = rd[5][b]
            want = np.take_along_axis(z, rd[3][b].astype(int)[:, None], 1)[:, 0] - z.max(-1) - np.log(np.exp(z - z.max(-1, keepdims=True)).sum(-1))
            assert np.all(np.abs(rd[6][b] - want) <= 2.0 ** -18)
        seq = np.concatenate([prompts[b]] + [rd[0][b, p].astype(int) for rd, p in zip(kept, steps)])
        part = slice(int(ends[b]) - n, int(ends[b]))
        q, k, v, dt, a = (np.concatenate([host(t[part])] + [rd[7 + i][b, p] for rd, p in zip(kept, steps)]) for i, t in enumerate(pin))
        m, xs = len(seq), host(table)[seq]
        o, mag, _ = op.conv(xs[:, :C], weight, bias, np.zeros((K - 1, C)))
        e = 1.1 * (K + 1) * E24 * mag + ((mag + 4) * 2.0 ** -23 + 2.0 ** -22) * np.abs(o)
        e = e + eps * (np.abs(o) + e)
        cut = lambda z: (z[:, H * P + G * N:].reshape(m, G, N), z[:, H * P:H * P + G * N].reshape(m, G, N), z[:, :H * P].reshape(m, H, P))  # noqa: E731
        for name, got, want, tol in zip("qkv", (q, k, v), cut(o), cut(e)):
            if rule and name != "v":
                s = N ** -0.5 if name == "q" else 1.0
                size = np.sqrt((want ** 2).sum(-1, keepdims=True) + 1e-6)
                row = np.sqrt((tol ** 2).sum(-1, keepdims=True)) / size
                assert row.max() < 0.1
                unit = op.unit(want, 1e-6, s)
                tol = 1.2 * (s * tol / size + row * np.abs(unit)) + ((N + 16) * E24 + eps) * (np.abs(unit) + s * tol / size)
                want = unit
            assert np.all(np.abs(got - want) <= tol), (b, name, float(np.max(np.abs(got - want) / tol)))
        if rule:
            beta, alpha = op.delta_gates(xs[:, C:C + H], xs[:, C + H:], dt_bias, a_log)
            assert np.all(np.abs(dt - beta) <= 2.0 ** -20 * beta) and np.all(np.abs(a - alpha) <= 2.0 ** -17 * alpha + 1e-37)
        scan, args = (op.delta_scan, (q, k, v, dt, a)) if rule else (op.scan, (q, k, v, dt, a))
        want, _ = scan(*args, np.zeros((H, P, N)))
        size = op.delta_size(*args, np.zeros((H, P, N)))[0] if rule else op.scan(*map(np.abs, args), np.zeros((H, P, N)))[0]
        tol = ((8 if rule else 1) * (3 * m + 2 * N + 128) * E24 + (2.0 ** -15 if io == "bf16" else 0)) * size
        outs = np.concatenate([rd[4][b, p] for rd, p in zip(kept, steps)])
        err = np.abs(outs - want[n:])
        assert np.all(err <= tol[n:]), (b, float(np.max(err / tol[n:])))
        err, tol = np.abs(host(py[part]) - want[:n]), tol[:n] + (2.0 ** -8 * np.abs(want[:n]) if io == "bf16" else 0)
        assert np.all(err <= tol), (b, float(np.max(err / tol)))
        assert int(layer.pos[b].item()) == sum(map(len, steps))
    assert B * rounds < accepted < B * rounds * W
    assert int(layer.base.min()) > 0   # flushed on the way
    layer.close()


@pytest.mark.parametrize("rule", [0, 1])
def test_two_layers_on_two_streams(rule):
    """Calls of two layers under way at once; each layer's outputs are those of the calls one after the other."""
    import linear_attention_decode_amd as lad
    gu.note(f"tree calls on two streams, rule {rule}")
    B, H, G, P, N, W, L = 5, 8, 2, 64, 128, 19, 16
    r = np.random.default_rng(4)
    dev = lambda a, t=torch.float32: torch.from_numpy(np.array(a)).to(t).to(gu.DEV)  # noqa: E731
    parent = dev([[-1 if w == 0 else int(r.integers(-1, w)) for w in range(W)] for _ in range(B)], torch.int32)

    def tokens(n):
        q, k = (op.unit(r.standard_normal((B, n, G, N)), 0) for _ in range(2))
        return (dev(q, torch.bfloat16), dev(k, torch.bfloat16), dev(r.standard_normal((B, n, H, P)), torch.bfloat16),
                dev(r.uniform(0, 1, (B, n, H))), dev(r.uniform(0.5, 1, (B, n, H))))
    layers, xs, ys = [], [], []
    for _ in range(2):
        layer = lad.ReplayLayer(B, H, G, P, N, L, io_dtype="bf16", rule="gdn" if rule else "mamba2", device=gu.DEV)
        layer.load_checkpoint(dev(0.5 * r.standard_normal((B, H, P, N))))
        layer.append(7, *tokens(7))
        layers.append(layer)
        xs.append(tokens(W))
        ys.append(torch.empty(3, B, W, H, P, device=gu.DEV))
    for i in range(2):
        layers[i].verify_tree(W, parent, *xs[i], ys[i][0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in (1, 2):
        for i in range(2):
            layers[i].verify_tree(W, parent, *xs[i], ys[i][turn], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ys[i][0], ys[i][1]) and torch.equal(ys[i][0], ys[i][2])
        assert bool(torch.isfinite(ys[i]).all()) and layers[i].get_error()[0] == 0
        layers[i].close()


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_captured_calls_on_changing_trees(rule, io):
    """One captured verification, replayed with other trees, counts and inputs, eager calls in between."""
    import linear_attention_decode_amd as lad
    gu.note(f"captured tree rule={rule} {io}")
    B, H, G, P, N, W, L, t_io = 4, 4, 2, 64, 64, 21, 32, torch.bfloat16 if io == "bf16" else torch.float32
    r = np.random.default_rng(9)
    dev = lambda a, t=torch.float32: torch.from_numpy(np.array(a)).to(t).to(gu.DEV)  # noqa: E731
    layer = lad.ReplayLayer(B, H, G, P, N, L, io_dtype=io, rule="gdn" if rule else "mamba2", device=gu.DEV)
    layer.load_checkpoint(dev(0.5 * r.standard_normal((B, H, P, N))))

    def tokens(n):
        q, k = (op.unit(r.standard_normal((B, n, G, N)), 0) for _ in range(2))
        return (dev(q, t_io), dev(k, t_io), dev(r.standard_normal((B, n, H, P)), t_io), dev(r.uniform(0, 1, (B, n, H))),
                dev(r.uniform(0.5, 1, (B, n, H))))
    tree = lambda: (dev([[-1 if w == 0 else int(r.integers(-1, w)) for w in range(W)] for _ in range(B)], torch.int32),  # noqa: E731
                    dev(r.integers(0, W + 1, B), torch.int32))
    parent, n = tree()
    xs, path, keep = tokens(W), torch.empty(B, W, dtype=torch.int32, device=gu.DEV), torch.empty(B, dtype=torch.int32, device=gu.DEV)
    fed, toks = (torch.zeros(B, W, dtype=torch.int32, device=gu.DEV) for _ in range(2))
    yg, ye = torch.zeros(B, W, H, P, device=gu.DEV), torch.zeros(B, W, H, P, device=gu.DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.verify_tree(W, parent, *xs, yg, n_nodes=n)
        lad.replay_accept_tree(parent, toks, fed, path, keep, n_nodes=n)
    for _ in range(6):
        layer.append(3, *tokens(3))
        layer.flush(L - 5)
        for dst, src in zip((parent, n, *xs), (*tree(), *tokens(W))):
            dst.copy_(src)
        for t in (fed, toks):
            t.copy_(dev(r.integers(0, 2, (B, W)), torch.int32))
        yg.fill_(7.0)
        ye.fill_(7.0)
        graph.replay()
        got = path.clone(), keep.clone()
        layer.verify_tree(W, parent, *xs, ye, n_nodes=n)
        lad.replay_accept_tree(parent, toks, fed, path, keep, n_nodes=n)
        torch.cuda.synchronize()
        assert torch.equal(yg, ye) and torch.equal(got[0], path) and torch.equal(got[1], keep)
        for b in range(B):
            assert bool((yg[b, int(n[b]):] == 7.0).all()) and not bool((yg[b, :int(n[b])] == 7.0).any())
    assert layer.get_error()[0] == 0
    layer.close()
