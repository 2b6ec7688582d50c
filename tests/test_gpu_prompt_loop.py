"""The prompt, token-input and sampling calls together, as a serving loop
uses them: prompts through the convolution and the scan into the layer, then
rounds of drafts -- convolution with the coming rollback, the fused round that
applies it, logits from its outputs, tokens and rejected drafts from these --
with nothing of the loop on the host but its launches.  Afterwards the float64
convolution and recurrence over the tokens that were accepted give the same
outputs for every one of them.

Bound: as for the scan, (3 n + N + 64) 2^-24 of the outputs' magnitudes for n
tokens, taken on the magnitudes of the convolution's sums, whose own
(K + 1) + 8 roundings enter q, k and v once each and dt once more: 64 more."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from oracle import runs
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H,G,P,N,K,lure", [([9, 1, 40], 4, 2, 64, 128, 4, 4.0), ([70, 33], 2, 1, 16, 16, 3, 4.0),
                                                 ([70, 33], 2, 1, 16, 16, 3, 1.0)])
def test_prompts_then_rounds_of_drafts(lens, H, G, P, N, K, lure):
    """lure: how much the logits favour the drafts; at 4 most are accepted, and all of the small heads'."""
    import linear_attention_decode_amd as lad
    gu.note(f"prompt loop {lens} P={P} N={N}")
    B, V, W, L, rounds = len(lens), 61, 4, 16, 12
    r = np.random.default_rng(sum(lens))
    C, f32, i32 = H * P + 2 * G * N, torch.float32, torch.int32
    dev = lambda a, t=f32: torch.from_numpy(np.array(a)).to(t).to(gu.DEV)  # noqa: E731
    # a row of the layer's projection for each token of the vocabulary, and the way back from its outputs
    table = r.standard_normal((V, C + H)).astype(np.float32)
    head = (r.standard_normal((H * P, V)) / np.sqrt(H * P)).astype(np.float32)
    weight, bias = r.uniform(-0.6, 0.6, (C, K)).astype(np.float32), r.uniform(-0.3, 0.3, C).astype(np.float32)
    dt_bias, a_log = r.uniform(-4, -1, H).astype(np.float32), np.log(r.uniform(1, 8, H)).astype(np.float32)
    conv = lad.ReplayConv(dev(weight), dev(bias), dev(dt_bias), dev(a_log), slots=K - 1 + W)
    layer = lad.ReplayLayer(B, H, G, P, N, L, io_dtype="f32", device=gu.DEV)
    rows, back = dev(table), dev(head)
    guess = lambda t: (t * 7 + 5) % V   # noqa: E731  what follows a token, in the drafts' opinion

    def logits(y, fed):   # the drafts are often right
        out = (y.reshape(-1, H * P) @ back).reshape(*fed.shape, V)
        return out.scatter_add(-1, guess(fed).long().unsqueeze(-1), torch.full((*fed.shape, 1), lure, device=gu.DEV)).contiguous()

    prompts = [r.integers(0, V, n) for n in lens]
    T, ends = sum(lens), np.cumsum(lens)
    x = rows[dev(np.concatenate(prompts), torch.long)]
    mk = lambda *s: (torch.empty(*s, G, N, device=gu.DEV), torch.empty(*s, G, N, device=gu.DEV),   # noqa: E731
                     torch.empty(*s, H, P, device=gu.DEV), torch.empty(*s, H, device=gu.DEV), torch.empty(*s, H, device=gu.DEV))
    cu, state = dev([0, *ends], i32), torch.empty(B, conv.slots, C, device=gu.DEV).fill_(float("nan"))
    ins = mk(T)
    layer.conv_prompt(conv, T, cu, x[:, :C], x[:, C:], None, state, *ins)
    y, S = torch.empty(T, H, P, device=gu.DEV), torch.empty(B, H, P, N, device=gu.DEV)
    need = lad.replay_scan_workspace(layer.cfg, T, max(lens))
    layer.scan(T, max(lens), cu, *ins, None, S, y, torch.empty(need, dtype=torch.uint8, device=gu.DEV) if need else None)
    layer.load_checkpoint(S)
    u = dev(r.uniform(0, 1, (rounds + 1, B, W)))
    settings = dict(temperature=dev([0.8] * B), top_k=dev([20] * B, i32), top_p=dev([0.95] * B), min_p=dev([0.01] * B))
    last = dev([p[-1] for p in prompts], i32).unsqueeze(1)
    token = torch.empty(B, 1, dtype=i32, device=gu.DEV)
    lad.replay_sample(logits(y[dev(ends - 1, torch.long)], last), u[rounds, :, :1].contiguous(), token, **settings)

    kept, nrej = [], None
    ins, outs = mk(B, W), torch.empty(B, W, H, P, device=gu.DEV)
    for rd in range(rounds):
        fed = [token]
        for _ in range(W - 1):
            fed.append(guess(fed[-1]))
        fed = torch.cat(fed, 1).contiguous()
        x = rows[fed.reshape(-1).long()]
        layer.conv_step(conv, W, x[:, :C], x[:, C:], state, *ins, n_reject=nrej)
        if nrej is None:
            layer.verify_step(W, *ins, outs)
        else:
            layer.rollback_verify_step(nrej, W, *ins, outs)
        tokens, nrej = torch.empty(B, W, dtype=i32, device=gu.DEV), torch.empty(B, dtype=i32, device=gu.DEV)
        lad.replay_sample(logits(outs, fed), u[rd].contiguous(), tokens, fed=fed, n_reject=nrej, **settings)
        token = tokens.gather(1, (W - 1 - nrej).long().unsqueeze(1))
        kept.append((fed, outs.clone(), nrej))
    torch.cuda.synchronize()
    assert layer.get_error()[0] == 0

    accepted = 0
    for b in range(B):
        stay = [int(W - n[b]) for _, _, n in kept]
        accepted += sum(stay)
        seq = np.concatenate([prompts[b]] + [f[b, :s].cpu().numpy() for (f, _, _), s in zip(kept, stay)])
        got = np.concatenate([y[ends[b] - lens[b]:ends[b]].cpu().numpy()] + [o[b, :s].cpu().numpy() for (_, o, _), s in zip(kept, stay)])
        n, xs = len(seq), table[seq].astype(np.float64)
        o, mag, _ = op.conv(xs[:, :C], weight, bias, np.zeros((K - 1, C)))
        dt, a = op.discretise(xs[:, C:], dt_bias, a_log)
        cut = lambda z: (z[:, H * P + G * N:].reshape(n, G, N), z[:, H * P:H * P + G * N].reshape(n, G, N), z[:, :H * P].reshape(n, H, P))  # noqa: E731
        want, _ = op.scan(*cut(o), dt, a, np.zeros((H, P, N)))
        size, _ = op.scan(*cut(1.1 * mag), dt, a, np.zeros((H, P, N)))
        tol = (3 * n + N + 128) * 2.0 ** -24 * size
        assert np.all(np.abs(got - want) <= tol), (b, float(np.max(np.abs(got - want) / tol)))
        assert int(layer.pos[b].item()) == sum(stay) + int(kept[-1][2][b])   # the last rollback is still to come
    assert B * rounds <= accepted <= B * rounds * W
    if lure == 4.0:
        assert accepted > B * rounds
    if lure == 1.0 or P == 64:
        assert accepted < B * rounds * W
    layer.close()


@pytest.mark.parametrize("lens,H,G", [([37, 1, 150], 128, 8), ([90, 65], 6, 2)])
def test_prompts_then_rounds_of_drafts_in_bf16(lens, H, G):
    """The same loop with bf16 io and 64 x 128 heads, the first one the decode benchmark's layer.

    The inputs that the convolution made are held to its own bound (its sums, then a rounding of 2^-8), the outputs to the
    float64 recurrence over these inputs: the prompt's, a float32 sum rounded to bf16, within ((3 n + N + 64) 2^-24 + 2^-15)
    of the sum of magnitudes and 2^-8 of itself; the rounds', float32, within the decode path's 1e-4 of a token's largest output."""
    import linear_attention_decode_amd as lad
    gu.note(f"prompt loop in bf16 {lens} H={H}")
    P, N, K, B, V, W, L, rounds, bf = 64, 128, 4, len(lens), 61, 4, 16, 8, torch.bfloat16
    r = np.random.default_rng(sum(lens) + H)
    C, f32, i32 = H * P + 2 * G * N, torch.float32, torch.int32
    dev = lambda a, t=f32: torch.from_numpy(np.array(a)).to(t).to(gu.DEV)  # noqa: E731
    rows, back = dev(r.standard_normal((V, C + H)), bf), dev(r.standard_normal((H * P, V)) / np.sqrt(H * P))
    weight, bias = r.uniform(-0.6, 0.6, (C, K)).astype(np.float32), r.uniform(-0.3, 0.3, C).astype(np.float32)
    dt_bias, a_log = r.uniform(-4, -1, H).astype(np.float32), np.log(r.uniform(1, 8, H)).astype(np.float32)
    conv = lad.ReplayConv(dev(weight), dev(bias), dev(dt_bias), dev(a_log), slots=K - 1 + W)
    layer = lad.ReplayLayer(B, H, G, P, N, L, io_dtype="bf16", device=gu.DEV)
    guess = lambda t: (t * 7 + 5) % V   # noqa: E731

    def logits(y, fed):
        out = (y.float().reshape(-1, H * P) @ back).reshape(*fed.shape, V)
        return out.scatter_add(-1, guess(fed).long().unsqueeze(-1), torch.full((*fed.shape, 1), 3.0, device=gu.DEV)).to(bf)

    mk = lambda *s: (*(torch.empty(*s, G, N, dtype=bf, device=gu.DEV) for _ in range(2)),   # noqa: E731
                     torch.empty(*s, H, P, dtype=bf, device=gu.DEV), *(torch.empty(*s, H, device=gu.DEV) for _ in range(2)))
    prompts, ends, T = [r.integers(0, V, n) for n in lens], np.cumsum(lens), sum(lens)
    cu, state, ins = dev([0, *ends], i32), torch.full((B, conv.slots, C), float("nan"), dtype=bf, device=gu.DEV), mk(T)
    x = rows[dev(np.concatenate(prompts), torch.long)]
    layer.conv_prompt(conv, T, cu, x[:, :C], x[:, C:], None, state, *ins)
    y, S = torch.empty(T, H, P, dtype=bf, device=gu.DEV), torch.empty(B, H, P, N, device=gu.DEV)
    need = lad.replay_scan_workspace(layer.cfg, T, max(lens))
    layer.scan(T, max(lens), cu, *ins, None, S, y, torch.empty(need, dtype=torch.uint8, device=gu.DEV) if need else None)
    layer.load_checkpoint(S)
    u = dev(r.uniform(0, 1, (rounds + 1, B, W)))
    settings = dict(temperature=dev([0.8] * B), top_k=dev([20] * B, i32), top_p=dev([0.95] * B), min_p=dev([0.01] * B))
    token = torch.empty(B, 1, dtype=i32, device=gu.DEV)
    lad.replay_sample(logits(y[dev(ends - 1, torch.long)], dev([p[-1] for p in prompts], i32).unsqueeze(1)),
                      u[rounds, :, :1].contiguous(), token, **settings)
    kept, nrej = [], None
    for rd in range(rounds):
        fed = [token]
        for _ in range(W - 1):
            fed.append(guess(fed[-1]))
        fed, win, out = torch.cat(fed, 1).contiguous(), mk(B, W), torch.empty(B, W, H, P, device=gu.DEV)
        x = rows[fed.reshape(-1).long()]
        layer.conv_step(conv, W, x[:, :C], x[:, C:], state, *win, n_reject=nrej)
        layer.verify_step(W, *win, out) if nrej is None else layer.rollback_verify_step(nrej, W, *win, out)
        tokens, nrej = torch.empty(B, W, dtype=i32, device=gu.DEV), torch.empty(B, dtype=i32, device=gu.DEV)
        lad.replay_sample(logits(out, fed), u[rd].contiguous(), tokens, fed=fed, n_reject=nrej, **settings)
        token = tokens.gather(1, (W - 1 - nrej).long().unsqueeze(1))
        kept.append((fed, win, out, nrej))
    torch.cuda.synchronize()
    assert layer.get_error()[0] == 0

    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    for b, n in enumerate(lens):
        stay = [int(W - k[3][b]) for k in kept]
        seq = np.concatenate([prompts[b]] + [host(k[0][b, :s]).astype(int) for k, s in zip(kept, stay)])
        part = slice(int(ends[b]) - n, int(ends[b]))
        q, k, v, dt, a = (np.concatenate([host(t[part])] + [host(w[1][i][b, :s]) for w, s in zip(kept, stay)])
                          for i, t in enumerate(ins))
        xs = host(rows)[seq]
        o, mag, _ = op.conv(xs[:, :C], weight, bias, np.zeros((K - 1, C)))
        got = np.concatenate([t.reshape(len(seq), -1) for t in (v, k, q)], 1)
        e = 1.1 * (K + 1) * 2.0 ** -24 * mag + ((mag + 4) * 2.0 ** -23 + 2.0 ** -22) * np.abs(o)
        assert np.all(np.abs(got - o) <= e + 2.0 ** -8 * (np.abs(o) + e))
        sums, _ = op.scan(q, k, v, dt, a, np.zeros((H, P, N)))
        size, _ = op.scan(np.abs(q[:n]), np.abs(k[:n]), np.abs(v[:n]), dt[:n], a[:n], np.zeros((H, P, N)))
        e = ((3 * n + N + 64) * 2.0 ** -24 + 2.0 ** -15) * size
        assert np.all(np.abs(host(y[part]) - sums[:n]) <= e + 2.0 ** -8 * (np.abs(sums[:n]) + e)), b
        outs = np.concatenate([host(w[2][b, :s]) for w, s in zip(kept, stay)])
        assert float(runs.normwise_rel_err(outs, sums[n:]).max()) <= 1e-4, b
        assert rounds <= sum(stay) <= rounds * W
    layer.close()
