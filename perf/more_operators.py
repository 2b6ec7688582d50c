"""What the Gated DeltaNet prompt, draft tree and token score operators do, case by case, in two forms: plain torch operations
and the library's calls.

Five operators of a serving loop around one SSM layer:

  delta_inputs  a Gated DeltaNet layer's q and k at unit length and its beta and alpha, from the convolution's outputs and the projection
  delta_scan    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T, y_t = S_t q_t over packed prompts, and the states
  conv_tree     the short causal convolution and the discretisation for a tree of drafted tokens, each node behind its ancestors
  verify_tree   outputs of a tree of drafted tokens against one read of the checkpoint and the ring
  logprobs      log-probabilities of given tokens, entropy and the most likely alternatives from logits

A case is a dict of plain values; `own` chooses the form.  Sequence lengths are a function of the case, values of the seed.
"""
import math
import random

import numpy as np
import torch

own = False

WIDTH = 4     # taps of the convolution
CHUNK = 64    # tokens of a chunk in the plain scan
EPS = 1e-6    # under the root of a row's length


# ---- cases -----------------------------------------------------------------

def _layer(batch, heads, groups, head_dim, state_dim, io):
    return {"batch": batch, "heads": heads, "groups": groups, "head_dim": head_dim, "state_dim": state_dim, "io": io}


def listed():
    return [
        # a few short prompts into a small float32 layer: launch latency counts
        {"name": "delta_scan_short_f32", "op": "delta_scan", **_layer(3, 4, 2, 64, 128, "f32"), "tokens": 97, "resume": False},
        # one long prompt alone on the card, the Gated DeltaNet benchmark's layer: 32 heads, chunk behind chunk
        {"name": "delta_scan_one_long", "op": "delta_scan", **_layer(1, 32, 16, 128, 128, "bf16"), "tokens": 8192, "resume": False},
        # a batch of ragged prompts that continue from states they left before (prompts taken in pieces)
        {"name": "delta_scan_batch_resumed", "op": "delta_scan", **_layer(16, 32, 16, 128, 128, "bf16"), "tokens": 15013, "resume": True},
        # the inputs of that batch, from rows of the layer's whole projection
        {"name": "delta_inputs_batch", "op": "delta_inputs", **_layer(16, 32, 16, 128, 128, "bf16"), "rows": 15013},
        # one token each of a small batch, float32, rows of an odd stride: latency
        {"name": "delta_inputs_step_f32", "op": "delta_inputs", **_layer(16, 5, 1, 64, 64, "f32"), "rows": 16},
        # the convolution of one sequence's drafts: latency
        {"name": "conv_tree_one", "op": "conv_tree", **_layer(1, 128, 8, 64, 128, "bf16"), "nodes": 16, "rule": 0},
        # the convolution of a batch's draft trees, at the verify benchmark's layer
        {"name": "conv_tree_batch", "op": "conv_tree", **_layer(256, 64, 8, 64, 128, "bf16"), "nodes": 16, "rule": 0},
        # one sequence's drafts: latency
        {"name": "verify_tree_one", "op": "verify_tree", **_layer(1, 128, 8, 64, 128, "bf16"), "nodes": 16, "ring": 16, "rule": 0,
         "read": "none"},
        # the verify benchmark's batch, a tree of 16 drafts in place of its window
        {"name": "verify_tree_batch", "op": "verify_tree", **_layer(256, 64, 8, 64, 128, "bf16"), "nodes": 16, "ring": 16, "rule": 0,
         "read": "none"},
        # large trees of a Gated DeltaNet layer, read from an e4m3 copy
        {"name": "verify_tree_delta", "op": "verify_tree", **_layer(96, 32, 16, 128, 128, "bf16"), "nodes": 41, "ring": 16, "rule": 1,
         "read": "fp8"},
        # one token of one sequence over a large vocabulary: latency
        {"name": "logprobs_one", "op": "logprobs", "batch": 1, "window": 1, "vocab": 131072, "io": "bf16", "given": 1, "top": 5,
         "tempered": False},
        # a batch's drafts and their bonus tokens, float32 logits of an odd vocabulary
        {"name": "logprobs_batch_f32", "op": "logprobs", "batch": 48, "window": 5, "vocab": 50021, "io": "f32", "given": 2, "top": 20,
         "tempered": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm, odd ones as likely as even ones."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["delta_scan", "delta_scan", "delta_inputs", "conv_tree", "verify_tree", "verify_tree", "logprobs"])
    if op == "logprobs":
        window = rng.choice([1, 1, 2, 5, 8])
        vocab = _spread(rng, 300, 200000)
        rows = _spread(rng, 1, max(1, min(1280, 256 * 131072 // vocab)))
        return {"op": op, "batch": max(1, rows // window), "window": window, "vocab": vocab, "io": rng.choice(["bf16", "f32"]),
                "given": rng.choice([0, 1, 1, 2, 7]), "top": rng.choice([0, 1, 5, 8, 20, 32]), "tempered": rng.random() < 0.5}
    P, N = rng.choice([(16, 16), (64, 64), (64, 128), (128, 128)])
    groups = rng.choice([1, 2, 8])
    heads = groups * _spread(rng, 1, 128 * 64 // (P * groups))
    c = _layer(0, heads, groups, P, N, rng.choice(["bf16", "bf16", "f32"]))
    if op == "delta_inputs":
        c["batch"] = _spread(rng, 1, 24)
        return {"op": op, **c, "rows": max(1, _spread(rng, 1, min(12000, 15013 * 16 * 128 // (groups * N))))}
    if op == "conv_tree":
        nodes = _spread(rng, 1, 64)
        c["batch"] = _spread(rng, 1, max(1, 2048 // nodes))
        return {"op": op, **c, "nodes": nodes, "rule": rng.choice([0, 0, 1])}
    if op == "verify_tree":
        nodes = _spread(rng, 1, 64)
        most = min(256 * 64 * 64 * 128 * 16 // (heads * P * N * max(16, nodes)), 16384 // heads)
        c["batch"] = _spread(rng, 1, max(1, most // (4 if c["io"] == "f32" else 2)))
        return {"op": op, **c, "nodes": nodes, "ring": rng.choice([5, 8, 16, 16, 32]), "rule": rng.choice([0, 1]),
                "read": rng.choice(["none", "none", "bf16", "fp8", "fp4"])}
    c["batch"] = _spread(rng, 1, 24)
    # no more work than the largest listed case: 15013 tokens of 32 heads of 128 x 128, a quarter of it in float32
    most = 15013 * 32 * 128 * 128 // (heads * P * N) // (8 if c["io"] == "f32" else 2)
    return {"op": op, **c, "tokens": max(c["batch"], _spread(rng, 1, min(12000, most))), "resume": rng.random() < 0.5}


def lengths(case):
    """Prompt lengths of a case: ragged, their sum the case's tokens, one of one token where there are several."""
    B, T = case["batch"], case["tokens"]
    rng = random.Random(B * 1000003 + T)
    weight = [rng.uniform(0.5, 1.5) for _ in range(B)]
    if B > 2:
        weight[B // 2] = 0.0
    cut = [0]
    for i in range(B):
        cut.append(round((T - B) * sum(weight[:i + 1]) / sum(weight)))
    return [cut[i + 1] - cut[i] + 1 for i in range(B)]


# ---- inputs ----------------------------------------------------------------

def _io(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _channels(case):
    return case["heads"] * case["head_dim"] + 2 * case["groups"] * case["state_dim"]


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # E2M1 values by code


def _copy_of(x, read):
    """A low-precision copy of the states x [B, H, P, N]: (codes, scales), as the layer keeps them."""
    B, H, P, N = x.shape
    if read == "bf16":
        return x.to(torch.bfloat16), None
    if read == "fp8":
        scale = x.abs().amax((2, 3)) / 448
        return (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale
    block = x.reshape(B, H, P * N // 32, 32)
    e = torch.floor(torch.log2(block.abs().amax(-1))) - 2
    z = block / torch.exp2(e).unsqueeze(-1)
    code = torch.bucketize(z.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)) + 8 * (z < 0)
    code = code.to(torch.uint8).reshape(B, H, P * N // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    s = {"case": dict(case)}
    if case["op"] == "logprobs":
        B, W, V, M, n = (case[x] for x in ("batch", "window", "vocab", "given", "top"))
        # a head's logits: a common slope over the vocabulary's ranks in a random order, and each position's own part
        rank = torch.argsort(torch.rand(V, generator=g, device="cuda")).float()
        s["logits"] = (normal(B, W, V) * 2.2 - 1.05 * torch.log(rank + 2.7)).to(_io(case))
        s["temperature"] = uniform(0.6, 1.2, B) if case["tempered"] else None
        # the tokens whose scores are asked: mostly likely ones, as a sampler draws them
        best = s["logits"].float().argmax(-1, keepdim=True).int()
        s["ids"] = torch.where(uniform(0, 1, B, W, M) < 0.4, best, whole(0, V, B, W, M)).contiguous() if M else None
        s["logp"] = torch.empty(B, W, M, device="cuda") if M else None
        s["entropy"] = torch.empty(B, W, device="cuda")
        s["top_ids"] = torch.empty(B, W, n, dtype=torch.int32, device="cuda") if n else None
        s["top_logp"] = torch.empty(B, W, n, device="cuda") if n else None
        return s

    B, H, G, P, N = (case[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    io = _io(case)
    act = torch.nn.functional.silu
    # step sizes between 0.001 and 0.1 at a zero projection, decay rates between 1 and 16
    dt0 = torch.exp(uniform(math.log(1e-3), math.log(0.1), H))
    dt_bias = dt0 + torch.log(-torch.expm1(-dt0))
    a_log = torch.log(uniform(1, 16, H))
    delta = case.get("rule", 1) == 1   # both scan and inputs are of Gated DeltaNet layers

    def tokens(*lead):
        """q, k, v, dt (beta), a (alpha) of the layer's kind."""
        q, k = act(normal(*lead, G, N)), act(normal(*lead, G, N))
        v = act(normal(*lead, H, P))
        dt = torch.nn.functional.softplus(normal(*lead, H) + dt_bias)
        a = torch.exp(-torch.exp(a_log) * dt)
        if delta:
            return (_unit(q) * N ** -0.5).to(io), _unit(k).to(io), v.to(io), torch.sigmoid(normal(*lead, H)), a
        return q.to(io), k.to(io), v.to(io), dt, a

    s["err"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    if case["op"] == "delta_scan":
        T = case["tokens"]
        s["cu"] = torch.tensor(np.cumsum([0] + lengths(case)).astype(np.int32)).cuda()
        s["q"], s["k"], s["v"], s["beta"], s["alpha"] = tokens(T)
        s["s_in"] = normal(B, H, P, N) * 0.3 if case["resume"] else None
        s["y"] = torch.empty(T, H, P, dtype=io, device="cuda")
        s["s_out"] = torch.empty(B, H, P, N, device="cuda")
        return s
    if case["op"] == "delta_inputs":
        T = case["rows"]
        s["q"], s["k"] = (act(normal(T, G, N)).to(io) for _ in range(2))
        # the layer's projection: [gate | v, k, q before the convolution | b | a]
        s["rows"] = normal(T, 2 * H * P + 2 * G * N + 2 * H).to(io)
        s["b_raw"], s["a_raw"] = s["rows"][:, -2 * H:-H], s["rows"][:, -H:]
        s["dt_bias"], s["a_log"] = dt_bias, a_log
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["beta"], s["alpha"] = (torch.empty(T, H, device="cuda") for _ in range(2))
        return s

    W = case["nodes"]
    # half the nodes carry on from the one before them, the others from any earlier one or from the sequence itself
    at = torch.arange(W, device="cuda", dtype=torch.int32).expand(B, W)
    other = (uniform(0, 1, B, W) * (at + 1)).int() - 1
    s["parent"] = torch.where(uniform(0, 1, B, W) < 0.5, at - 1, torch.minimum(other, at - 1)).contiguous()
    # the trees of a batch differ in size
    s["n_nodes"] = torch.where(uniform(0, 1, B) < 0.7, torch.full((B,), W, device="cuda", dtype=torch.int32), whole(0, W + 1, B))
    if case["op"] == "conv_tree":
        C, R = _channels(case), WIDTH - 1 + 16
        s["weight"] = uniform(-0.5, 0.5, C, WIDTH)
        s["bias"] = uniform(-0.5, 0.5, C)
        s["dt_bias"], s["a_log"] = dt_bias, a_log
        s["state"] = normal(B, R, C).to(io)
        s["pos"] = whole(8, 5000, B)
        s["rows"] = normal(B * W, H * P + C + H).to(io)
        s["x"] = s["rows"][:, H * P:H * P + C]
        s["dt_raw"] = None if delta else s["rows"][:, H * P + C:]
        s["q"], s["k"] = (torch.zeros(B, W, G, N, dtype=io, device="cuda") for _ in range(2))
        s["v"] = torch.zeros(B, W, H, P, dtype=io, device="cuda")
        s["dt"], s["a"] = (None if delta else torch.zeros(B, W, H, device="cuda") for _ in range(2))
        return s

    L = case["ring"]
    s["q"], s["k"], s["v"], s["dt"], s["a"] = tokens(B, W)
    _, k, v, dt, a = tokens(B, L)
    s["ring_k"], s["ring_v"] = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
    s["ring_dt"], s["ring_a"] = dt, a
    s["base"] = whole(0, 5000, B)
    s["pos"] = s["base"] + whole(0, L + 1, B)
    state = normal(B, H, P, N) * 0.3
    if case["read"] == "none":
        s["master"] = state
    else:
        s["copy"], s["scale"] = _copy_of(state, case["read"])
    s["y"] = torch.zeros(B, W, H, P, device="cuda")
    return s


# ---- the plain forms -------------------------------------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_delta_inputs(s):
    N = s["case"]["state_dim"]
    alpha = torch.exp(-torch.exp(s["a_log"]) * _softplus(s["a_raw"].float() + s["dt_bias"]))
    return {"q": (_unit(s["q"].float()) * N ** -0.5).to(s["q"].dtype), "k": _unit(s["k"].float()).to(s["k"].dtype),
            "beta": 1 / (1 + torch.exp(-s["b_raw"].float())), "alpha": alpha}


def _solved(A):
    """(I + A)^-1 of strictly lower triangular A, row by row."""
    n = A.shape[-1]
    X = torch.eye(n, device=A.device).expand(A.shape).clone()
    for i in range(1, n):
        X[..., i, :i] = -(A[..., i, None, :i] @ X[..., :i, :i]).squeeze(-2)
    return X


def _plain_delta_scan(s):
    c = s["case"]
    B, H, G, P, N = (c[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    Q, R, io = CHUNK, H // G, s["y"].dtype
    nc = -(-max(lengths(c)) // Q)
    cu = s["cu"].long()
    at = torch.arange(nc * Q, device=cu.device)
    there = at < (cu[1:] - cu[:-1]).unsqueeze(1)
    row = torch.where(there, cu[:-1].unsqueeze(1) + at, 0)

    def chunks(t, heads, width):   # [B, nc, heads, Q, width], zero past a sequence's end
        return torch.where(there[..., None, None], t.float()[row], 0).view(B, nc, Q, heads, width).transpose(2, 3)

    q, k, v = chunks(s["q"], G, N), chunks(s["k"], G, N), chunks(s["v"], H, P)
    beta = torch.where(there.unsqueeze(-1), s["beta"][row], 0).view(B, nc, Q, H).transpose(2, 3)
    alpha = torch.where(there.unsqueeze(-1), s["alpha"][row], 1).view(B, nc, Q, H).transpose(2, 3)
    csum = torch.cumsum(torch.log(alpha.double()), -1)                    # [B, nc, H, Q]
    lower = torch.ones(Q, Q, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp(torch.where(lower, csum.unsqueeze(-1) - csum.unsqueeze(-2), -math.inf).float())
    each = lambda t: t.repeat_interleave(R, 2)  # noqa: E731  a group's rows for each of its heads
    solve = _solved((each(k @ k.transpose(-1, -2)) * decay * beta.unsqueeze(-1)).tril(-1)) * beta.unsqueeze(-2)
    score = each(q @ k.transpose(-1, -2)) * decay
    into = torch.exp(csum.float()).unsqueeze(-1)
    last = torch.exp((csum[..., -1:] - csum).float()).unsqueeze(-1)
    S = torch.zeros(B, H, P, N, device=q.device) if s["s_in"] is None else s["s_in"]
    y = torch.empty(B, nc, H, Q, P, device=q.device)
    for i in range(nc):
        ki, qi = k[:, i].repeat_interleave(R, 1), q[:, i].repeat_interleave(R, 1)
        u = solve[:, i] @ (v[:, i] - into[:, i] * (ki @ S.transpose(-1, -2)))
        y[:, i] = into[:, i] * (qi @ S.transpose(-1, -2)) + score[:, i] @ u
        S = into[:, i, :, -1:] * S + (u * last[:, i]).transpose(-1, -2) @ ki
    return {"y": y.transpose(2, 3).reshape(B, nc * Q, H, P)[there].to(io), "s_out": S.clone()}


def _behind(parent, steps):
    """Each node's ancestor that many steps up (itself at 0), and how many steps past its root the others are: [B, W] pairs."""
    B, W = parent.shape
    parent = torch.cat([parent.long(), torch.full((B, 1), -1, device=parent.device)], 1)   # past the roots: index W
    node = torch.arange(W, device=parent.device).expand(B, W)
    past = torch.zeros(B, W, dtype=torch.long, device=parent.device)
    out = [(node, past)]
    for _ in range(steps):
        up = parent.gather(1, node)
        past = past + (up < 0)
        node = torch.where(up < 0, W, up)
        out.append((node, past))
    return out


def _plain_conv_tree(s):
    c = s["case"]
    B, W, H, G, P, N, K = c["batch"], c["nodes"], c["heads"], c["groups"], c["head_dim"], c["state_dim"], WIDTH
    io, R = s["q"].dtype, s["state"].shape[1]
    there = torch.arange(W, device=s["x"].device) < s["n_nodes"].unsqueeze(1)
    seq = torch.arange(B, device=s["x"].device).unsqueeze(1)
    x = torch.cat([s["x"].float().view(B, W, -1), torch.zeros(B, 1, s["x"].shape[1], device=s["x"].device)], 1)
    acc = s["bias"].expand(B, W, -1)
    for d, (node, past) in enumerate(_behind(s["parent"], K - 1)):
        old = s["state"][seq, (s["pos"].long().unsqueeze(1) - past) % R].float()
        acc = acc + s["weight"][:, K - 1 - d] * torch.where((past > 0).unsqueeze(-1), old, x[seq, node])
    o = torch.where(there.unsqueeze(-1), _silu(acc), 0).to(io)
    v, k, q = torch.split(o, [H * P, G * N, G * N], -1)
    out = {"v": v.reshape(B, W, H, P), "k": k.reshape(B, W, G, N), "q": q.reshape(B, W, G, N)}
    if s["dt_raw"] is not None:
        dt = _softplus(s["dt_raw"].float() + s["dt_bias"]).view(B, W, H)
        out["dt"] = torch.where(there.unsqueeze(-1), dt, 0)
        out["a"] = torch.where(there.unsqueeze(-1), torch.exp(-torch.exp(s["a_log"]) * dt), 0)
    return out


def _checkpoint(s):
    """The state that the outputs read, [B, H, P, N] float32."""
    c = s["case"]
    if c["read"] == "none":
        return s["master"]
    if c["read"] == "bf16":
        return s["copy"].float()
    if c["read"] == "fp8":
        return s["copy"].view(torch.float8_e4m3fn).float() * s["scale"][..., None, None]
    value = torch.tensor(FP4 + tuple(-x for x in FP4), device=s["copy"].device)
    code = torch.stack([s["copy"] & 15, s["copy"] >> 4], -1).long()
    shape = (c["batch"], c["heads"], c["head_dim"], c["state_dim"])
    x = value[code].view(*shape[:2], -1, 32) * torch.exp2(s["scale"].float() - 127).unsqueeze(-1)
    return x.view(shape)


def _entries(s):
    """The ring's entries, oldest first, and the nodes behind them: k, v, dt, a [B, L + W, ...], and the parent of each
    among them (an entry that is not there: behind nothing, without weight)."""
    c = s["case"]
    B, L, W = c["batch"], c["ring"], c["nodes"]
    dev = s["parent"].device
    count = (s["pos"] - s["base"]).long()
    seq, j = torch.arange(B, device=dev).unsqueeze(1), torch.arange(L, device=dev)
    slot = (s["base"].long().unsqueeze(1) + j) % L
    node = torch.arange(W, device=dev) < s["n_nodes"].unsqueeze(1)
    there = torch.cat([j < count.unsqueeze(1), node], 1)
    k = torch.cat([s["ring_k"].transpose(1, 2)[seq, slot], s["k"]], 1).float()
    v = torch.cat([s["ring_v"].transpose(1, 2)[seq, slot], s["v"]], 1).float()
    k, v = (torch.where(there[..., None, None], t, 0) for t in (k, v))
    dt = torch.where(there.unsqueeze(-1), torch.cat([s["ring_dt"][seq, slot], s["dt"]], 1), 0)
    a = torch.where(there.unsqueeze(-1), torch.cat([s["ring_a"][seq, slot], s["a"]], 1), 1)
    up = torch.where(node, s["parent"].long(), -1)
    up = torch.cat([(j - 1).expand(B, L), torch.where(up < 0, L - 1, up + L)], 1)
    return k, v, dt, a, up, node


def _plain_verify_tree(s):
    c = s["case"]
    B, W, L, R = c["batch"], c["nodes"], c["ring"], c["heads"] // c["groups"]
    k, v, dt, a, up, node = _entries(s)
    E = L + W
    S = _checkpoint(s)
    # anc[b, i, j]: j is i or lies on the way to it; path: the logarithm of the decays up to and with i
    anc = torch.zeros(B, E, E, dtype=torch.bool, device=S.device)
    path = torch.log(a.double()).transpose(1, 2)                        # [B, H, E]
    seq = torch.arange(B, device=S.device)
    for i in range(E):
        if i:
            anc[:, i] = anc[seq, up[:, i]]
            path[:, :, i] += path.gather(2, up[:, i].view(B, 1, 1).expand(B, c["heads"], 1)).squeeze(-1)
        anc[:, i, i] = True
    heads = lambda t: t.transpose(1, 2).repeat_interleave(R, 1)  # noqa: E731  [B, H, ., N] of [B, ., G, N]
    kh, qh, vh, dth = heads(k), heads(s["q"].float()), v.transpose(1, 2), dt.transpose(1, 2)
    decay = torch.exp(torch.where(anc.unsqueeze(1), path.unsqueeze(-1) - path.unsqueeze(-2), -math.inf).float())   # [B, H, E, E]
    into = torch.exp(path.float()).unsqueeze(-1)
    St = S.transpose(-1, -2)
    if c["rule"] == 1:
        A = ((kh @ kh.transpose(-1, -2)) * decay * dth.unsqueeze(-1)).tril(-1)
        u = _solved(A) @ (dth.unsqueeze(-1) * (vh - into * (kh @ St)))
    else:
        u = dth.unsqueeze(-1) * vh
    y = into[:, :, L:] * (qh @ St) + ((qh @ kh.transpose(-1, -2)) * decay[:, :, L:]) @ u
    return {"y": torch.where(node[..., None, None], y.transpose(1, 2), 0)}


def _plain_logprobs(s):
    n = s["case"]["top"]
    x = s["logits"].double()
    if s["temperature"] is not None:
        x = x / s["temperature"].double().view(-1, 1, 1)
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    Z = e.sum(-1, keepdim=True)
    out = {"entropy": (torch.log(Z) - (e * x).sum(-1, keepdim=True) / Z).squeeze(-1).float()}
    x = x - torch.log(Z)
    if s["ids"] is not None:
        out["logp"] = x.gather(-1, s["ids"].long()).float()
    if n:
        order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)[1][..., :n]
        out["top_ids"], out["top_logp"] = order.int(), x.gather(-1, order).float()
    return out


# ---- the library's calls ---------------------------------------------------

def _kept(s):
    """What a serving program keeps from call to call: the layer, its convolution, a workspace."""
    import linear_attention_decode_amd as lad
    if "kept" not in s:
        c, kept, need = s["case"], {}, 0
        if c["op"] == "logprobs":
            need = lad.replay_logprobs_workspace(c["batch"], c["window"], c["vocab"], c["top"])
        elif c["op"] == "verify_tree":
            layer = lad.ReplayLayer(c["batch"], c["heads"], c["groups"], c["head_dim"], c["state_dim"], c["ring"], io_dtype=c["io"],
                                    read_copy=None if c["read"] == "none" else c["read"], rule="gdn" if c["rule"] else "mamba2")
            for mine, theirs in (("master", "s_master"), ("copy", "s_copy"), ("scale", "s_scale"), ("ring_k", "ring_k"),
                                 ("ring_v", "ring_v"), ("ring_dt", "ring_dt"), ("ring_a", "ring_a"), ("base", "base"), ("pos", "pos")):
                if s.get(mine) is not None:
                    layer.t[theirs].copy_(s[mine])
            layer.set_flush_skipping(False)
            kept["layer"] = layer
        else:
            kept["cfg"] = lad.ReplayConfig(c["batch"], c["heads"], c["groups"], c["head_dim"], c["state_dim"], 16,
                                           lad.BF16 if c["io"] == "bf16" else lad.F32, lad.NONE, 0, c.get("rule", 1))
            if c["op"] == "delta_scan":
                kept["most"] = max(lengths(c))
                need = lad.replay_delta_scan_workspace(kept["cfg"], c["tokens"], kept["most"])
            elif c["op"] == "conv_tree":
                kept["conv"] = lad.ReplayConv(s["weight"], s["bias"], s["dt_bias"], s["a_log"], slots=s["state"].shape[1])
        kept["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        s["kept"] = kept
    return lad, s["kept"]


def _own(s):
    lad, kept = _kept(s)
    c = s["case"]
    if c["op"] == "delta_scan":
        lad.replay_delta_scan(kept["cfg"], c["tokens"], kept["most"], s["cu"], s["q"], s["k"], s["v"], s["beta"], s["alpha"],
                              s["s_in"], s["s_out"], s["y"], s["err"], kept["workspace"])
        return {"y": s["y"], "s_out": s["s_out"]}
    if c["op"] == "delta_inputs":
        lad.replay_delta_inputs(kept["cfg"], c["rows"], s["q"], s["k"], s["b_raw"], s["a_raw"], s["dt_bias"], s["a_log"],
                                c["state_dim"] ** -0.5, EPS, s["q_out"], s["k_out"], s["beta"], s["alpha"])
        return {"q": s["q_out"], "k": s["k_out"], "beta": s["beta"], "alpha": s["alpha"]}
    if c["op"] == "conv_tree":
        lad.replay_conv_tree(kept["cfg"], kept["conv"], c["nodes"], s["parent"], s["x"], s["dt_raw"], s["pos"], s["state"],
                             s["q"], s["k"], s["v"], s["dt"], s["a"], s["err"], n_nodes=s["n_nodes"])
        return {n: s[n] for n in ("v", "k", "q", "dt", "a") if s[n] is not None}
    if c["op"] == "verify_tree":
        kept["layer"].verify_tree(c["nodes"], s["parent"], s["q"], s["k"], s["v"], s["dt"], s["a"], s["y"], n_nodes=s["n_nodes"])
        return {"y": s["y"]}
    lad.replay_logprobs(s["logits"], ids=s["ids"], logp=s["logp"], entropy=s["entropy"], top_ids=s["top_ids"],
                        top_logp=s["top_logp"], temperature=s["temperature"], workspace=kept["workspace"])
    return {n: s[n] for n in ("entropy", "logp", "top_ids", "top_logp") if s[n] is not None}


def run(state):
    if own:
        return _own(state)
    return {"delta_scan": _plain_delta_scan, "delta_inputs": _plain_delta_inputs, "conv_tree": _plain_conv_tree,
            "verify_tree": _plain_verify_tree, "logprobs": _plain_logprobs}[state["case"]["op"]](state)


# ---- what a pass cannot do without, and what it should give ------------------

def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "logprobs":
        rows = case["batch"] * case["window"]
        # the logits once; a comparison, a difference, an exponential and two sums each
        return {"bytes": rows * (case["vocab"] * e + 8 * case["given"] + 8 * case["top"] + 4), "flops": 6 * rows * case["vocab"]}
    B, H, G, P, N = (case[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    if case["op"] == "delta_scan":
        T = case["tokens"]
        states = B * H * P * N * 4 * (2 if case["resume"] else 1)
        # v, y, q, k, beta and alpha once, and the states; S k and S q out of the state, u k^T into it
        return {"bytes": T * (2 * H * P * e + 2 * G * N * e + 8 * H) + states, "flops": 6 * T * H * P * N}
    if case["op"] == "delta_inputs":
        T = case["rows"]
        return {"bytes": T * (4 * G * N * e + 2 * H * (e + 4)) + 8 * H, "flops": T * (8 * G * N + 20 * H)}
    W, C = case["nodes"], _channels(case)
    if case["op"] == "conv_tree":
        gate = 0 if case["rule"] else H * (e + 8)
        return {"bytes": B * W * (2 * C * e + gate + 4) + B * (WIDTH - 1) * C * e + C * (WIDTH + 1) * 4,
                "flops": B * W * C * (2 * WIDTH + 4)}
    state = {"none": 4, "bf16": 2, "fp8": 1, "fp4": 17 / 32}[case["read"]]
    half = case["ring"] // 2 + W   # entries: a ring is half full on average
    return {"bytes": int(B * H * P * N * state) + B * half * (G * N * e + H * P * e + 8 * H) + B * W * (G * N * e + 4 * H * P),
            "flops": 2 * B * W * (H * P * N + half * (G * N + H * P))}


def _exact_delta_scan(case, s):
    """The recurrence itself, token after token in 64 bits, all sequences side by side."""
    B, H, G, P, N = (case[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    lens = lengths(case)
    first = np.cumsum([0] + lens)
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda") if s["s_in"] is None else s["s_in"].double()
    y = torch.zeros(case["tokens"], H, P, dtype=torch.float64, device="cuda")
    # the longest first: the sequences that still run are the first ones
    by = sorted(range(B), key=lambda b: -lens[b])
    S = S[by].contiguous()
    for i in range(lens[by[0]]):
        n = sum(lens[b] > i for b in by)
        row = torch.tensor([int(first[b]) + i for b in by[:n]]).cuda(non_blocking=True)
        k, q = (s[m][row].double().repeat_interleave(H // G, 1).unsqueeze(-2) for m in ("k", "q"))
        S[:n].mul_(s["alpha"][row].double()[..., None, None])
        miss = s["v"][row].double() - (S[:n] * k).sum(-1)
        S[:n].add_((miss * s["beta"][row].double().unsqueeze(-1)).unsqueeze(-1) * k)
        y[row] = (S[:n] * q).sum(-1)
    out = torch.empty_like(S)
    out[by] = S
    return {"y": y, "s_out": out}


def _exact_delta_inputs(case, s):
    def unit(t):
        t = t.double()
        return t * torch.rsqrt(torch.linalg.vecdot(t, t).unsqueeze(-1) + EPS)

    raw = s["a_raw"].double() + s["dt_bias"].double()
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    return {"q": unit(s["q"]) / math.sqrt(case["state_dim"]), "k": unit(s["k"]), "beta": torch.sigmoid(s["b_raw"].double()),
            "alpha": torch.exp(-torch.exp(s["a_log"].double()) * step)}


def _exact_conv_tree(case, s):
    """Node after node in 64 bits: the three rows before a node are those before its parent, moved on by the parent's."""
    B, W, H, G, P, N = (case[n] for n in ("batch", "nodes", "heads", "groups", "head_dim", "state_dim"))
    R, C = s["state"].shape[1], _channels(case)
    seq = torch.arange(B, device="cuda")
    x = s["x"].double().view(B, W, C)
    before = torch.zeros(B, W + 1, WIDTH - 1, C, dtype=torch.float64, device="cuda")   # at W: before a root
    for i in range(1, WIDTH):
        before[:, W, WIDTH - 1 - i] = s["state"][seq, (s["pos"].long() - i) % R].double()
    sums = torch.empty(B, W, C, dtype=torch.float64, device="cuda")
    for w in range(W):
        up = s["parent"][:, w].long()
        root = (up < 0).view(B, 1, 1)
        moved = torch.cat([before[seq, up.clamp(min=0)][:, 1:], x[seq, up.clamp(min=0)].unsqueeze(1)], 1)
        before[:, w] = torch.where(root, before[:, W], moved)
        rows = torch.cat([before[:, w], x[:, w:w + 1]], 1)
        sums[:, w] = (rows * s["weight"].double().t()).sum(1) + s["bias"].double()
    there = (torch.arange(W, device="cuda") < s["n_nodes"].unsqueeze(1)).unsqueeze(-1)
    o = torch.where(there, sums * torch.sigmoid(sums), 0)
    out = {"v": o[..., :H * P].reshape(B, W, H, P), "k": o[..., H * P:H * P + G * N].reshape(B, W, G, N),
           "q": o[..., H * P + G * N:].reshape(B, W, G, N)}
    if s["dt_raw"] is not None:
        raw = s["dt_raw"].double() + s["dt_bias"].double()
        dt = torch.logaddexp(raw, torch.zeros_like(raw)).view(B, W, H)
        out["dt"] = torch.where(there, dt, 0)
        out["a"] = torch.where(there, torch.exp(-torch.exp(s["a_log"].double()) * dt), 0)
    return out


def _exact_verify_tree(case, s):
    """Every node's state from its parent's, in 64 bits, a few sequences at a time."""
    B, W, L, H, G, P, N = (case[n] for n in ("batch", "nodes", "ring", "heads", "groups", "head_dim", "state_dim"))
    read = _checkpoint(s)
    y = torch.zeros(B, W, H, P, dtype=torch.float64, device="cuda")

    def step(S, k, v, dt, a):   # k [b, G, N], v [b, H, P], dt, a [b, H]
        k = k.double().repeat_interleave(H // G, 1).unsqueeze(-2)
        S = S * a.double()[..., None, None]
        add = v.double()
        if case["rule"]:
            add = add - (S * k).sum(-1)
        return S + (add * dt.double().unsqueeze(-1)).unsqueeze(-1) * k

    some = max(1, 2 ** 28 // ((W + 1) * H * P * N))
    for b0 in range(0, B, some):
        b = torch.arange(b0, min(B, b0 + some), device="cuda")
        S = read[b].double()
        count = (s["pos"] - s["base"])[b]
        for j in range(L):
            slot = (s["base"][b].long() + j) % L
            after = step(S, s["ring_k"][b, :, slot], s["ring_v"][b, :, slot], s["ring_dt"][b, slot], s["ring_a"][b, slot])
            S = torch.where((j < count).view(-1, 1, 1, 1), after, S)
        tree = torch.empty(len(b), W + 1, H, P, N, dtype=torch.float64, device="cuda")
        tree[:, 0] = S
        at = torch.arange(len(b), device="cuda")
        for w in range(W):
            tree[:, w + 1] = step(tree[at, s["parent"][b, w].long() + 1], s["k"][b, w], s["v"][b, w], s["dt"][b, w], s["a"][b, w])
            q = s["q"][b, w].double().repeat_interleave(H // G, 1).unsqueeze(-2)
            out = (tree[:, w + 1] * q).sum(-1)
            y[b, w] = torch.where((w < s["n_nodes"][b]).view(-1, 1, 1), out, 0)
    return {"y": y}


def _exact_logprobs(case, s):
    """Row by row on the host in 64-bit floating point."""
    B, W, M, n = (case[x] for x in ("batch", "window", "given", "top"))
    out = {"entropy": np.zeros((B, W))}
    if M:
        out["logp"] = np.zeros((B, W, M))
    if n:
        out["top_logp"] = np.zeros((B, W, n))
    T = np.ones(B) if s["temperature"] is None else s["temperature"].double().cpu().numpy()
    for b in range(B):
        for w, x in enumerate(s["logits"][b].double().cpu().numpy()):
            x = x / T[b]
            lp = x - (x.max() + np.log(np.exp(x - x.max()).sum()))
            out["entropy"][b, w] = -(np.exp(lp) * lp).sum()
            if M:
                out["logp"][b, w] = lp[s["ids"][b, w].cpu().numpy()]
            if n:
                out["top_logp"][b, w] = -np.sort(-lp)[:n]
    out = {name: torch.from_numpy(t) for name, t in out.items()}
    if n:
        out["top_ids"] = None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta_scan": _exact_delta_scan, "delta_inputs": _exact_delta_inputs, "conv_tree": _exact_conv_tree,
            "verify_tree": _exact_verify_tree, "logprobs": _exact_logprobs}[case["op"]](case, s)
