"""What the prompt and sampling operators do, case by case, in two forms: plain torch operations and the library's calls.

Four operators of a serving loop around one SSM layer:

  conv_prompt  the short causal convolution and the discretisation that turn a prompt batch's projected rows into (q, k, v, dt, a)
  conv_step    the same for one token, or a window of drafts, per sequence
  scan         S_t = a_t S_{t-1} + dt_t v_t k_t^T, y_t = S_t q_t over packed prompts, and the state that they leave
  sample       tokens from logits by temperature, top-k, top-p and min-p with given random numbers, and the rejected drafts

A case is a dict of plain values; `own` chooses the form.  Sequence lengths are a function of the case, values of the seed.
"""
import math
import random

import numpy as np
import torch

own = False

WIDTH = 4          # taps of the convolution
CHUNK = 64         # tokens of a chunk in the plain scan
ONE = float(2 ** 45)   # weight of the largest logit in `sample`


# ---- cases -----------------------------------------------------------------

def _layer(batch, heads, groups, head_dim, state_dim, io):
    return {"batch": batch, "heads": heads, "groups": groups, "head_dim": head_dim, "state_dim": state_dim, "io": io}


def listed():
    return [
        # a few short prompts into a small float32 layer: launch latency counts
        {"name": "scan_short_f32", "op": "scan", **_layer(3, 4, 2, 64, 128, "f32"), "tokens": 97, "resume": False},
        # one long prompt alone on the card, the decode benchmark's layer: the sequence has to be split to fill it
        {"name": "scan_one_long", "op": "scan", **_layer(1, 128, 8, 64, 128, "bf16"), "tokens": 8192, "resume": False},
        # a batch of ragged prompts that continue from states they left before (a prompt taken in pieces)
        {"name": "scan_batch_resumed", "op": "scan", **_layer(16, 128, 8, 64, 128, "bf16"), "tokens": 15013, "resume": True},
        # 128 x 128 heads in float32, odd lengths
        {"name": "scan_wide_f32", "op": "scan", **_layer(4, 32, 8, 128, 128, "f32"), "tokens": 1999, "resume": True},
        # the convolution of the ragged batch above, from rows of the layer's whole projection
        {"name": "conv_prompt_batch", "op": "conv_prompt", **_layer(16, 128, 8, 64, 128, "bf16"), "tokens": 15013, "resume": False},
        # short float32 prompts, an odd number of heads: rows of an odd stride
        {"name": "conv_prompt_odd_f32", "op": "conv_prompt", **_layer(3, 5, 1, 64, 64, "f32"), "tokens": 203, "resume": True},
        # one token of one sequence: latency
        {"name": "conv_step_one", "op": "conv_step", **_layer(1, 128, 8, 64, 128, "bf16"), "window": 1, "rollback": False},
        # one token each of the decode benchmark's batch
        {"name": "conv_step_batch", "op": "conv_step", **_layer(256, 128, 8, 64, 128, "bf16"), "window": 1, "rollback": False},
        # a window of drafts each, the last round's rejected drafts still to be dropped
        {"name": "conv_step_verify", "op": "conv_step", **_layer(256, 64, 8, 64, 128, "bf16"), "window": 5, "rollback": True},
        # one token for one sequence over a large vocabulary: latency
        {"name": "sample_one", "op": "sample", "batch": 1, "window": 1, "vocab": 131072, "io": "bf16", "filters": "all"},
        # the decode benchmark's batch, every filter in use
        {"name": "sample_batch", "op": "sample", "batch": 256, "window": 1, "vocab": 131072, "io": "bf16", "filters": "all"},
        # windows of drafts: float32 logits of an odd vocabulary, accepted against the tokens that were fed
        {"name": "sample_verify", "op": "sample", "batch": 48, "window": 5, "vocab": 50021, "io": "f32", "filters": "mixed"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm, odd ones as likely as even ones."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "conv_prompt", "conv_step", "sample"])
    if op == "sample":
        window = rng.choice([1, 1, 2, 5, 8])
        vocab = _spread(rng, 300, 200000)
        rows = _spread(rng, 1, max(1, min(1280, 256 * 131072 // vocab)))
        return {"op": op, "batch": max(1, rows // window), "window": window, "vocab": vocab, "io": rng.choice(["bf16", "f32"]),
                "filters": rng.choice(["all", "mixed", "none"])}
    P, N = rng.choice([(16, 16), (64, 64), (64, 128), (128, 128)])
    groups = rng.choice([1, 2, 8])
    heads = groups * _spread(rng, 1, 128 * 64 // (P * groups))
    c = _layer(0, heads, groups, P, N, rng.choice(["bf16", "bf16", "f32"]))
    if op == "conv_step":
        window = rng.choice([1, 1, 2, 5, 8])
        c["batch"] = _spread(rng, 1, max(1, 256 // window))
        return {"op": op, **c, "window": window, "rollback": rng.random() < 0.5}
    c["batch"] = _spread(rng, 1, 24)
    # no more work than the largest listed case: 15013 tokens of 128 heads of 64 x 128, a quarter of it in float32
    most = 15013 * 128 * 64 * 128 // (heads * P * N) // (8 if c["io"] == "f32" else 2)
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


def _cu(case):
    return torch.tensor(np.cumsum([0] + lengths(case)).astype(np.int32)).cuda()


def _channels(case):
    return case["heads"] * case["head_dim"] + 2 * case["groups"] * case["state_dim"]


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
    if case["op"] == "sample":
        B, W, V = case["batch"], case["window"], case["vocab"]
        # a head's logits: a common slope over the vocabulary's ranks in a random order, and each position's own part
        rank = torch.argsort(torch.rand(V, generator=g, device="cuda")).float()
        s["logits"] = (normal(B, W, V) * 2.2 - 1.05 * torch.log(rank + 2.7)).to(_io(case))
        s["u"] = uniform(0, 1, B, W)
        pick = uniform(0, 1, 4, B)
        some = case["filters"] == "mixed"
        if case["filters"] != "none":
            s["temperature"] = torch.where(pick[0] < (0.15 if some else 0.0), 0.0, uniform(0.6, 1.2, B))
            s["top_k"] = torch.where(pick[1] < (0.4 if some else 0.0), 0, whole(1, min(V, 1000), B))
            s["top_p"] = torch.where(pick[2] < (0.4 if some else 0.0), 1.0, uniform(0.8, 0.98, B))
            s["min_p"] = torch.where(pick[3] < (0.6 if some else 0.0), 0.0, uniform(0.0, 0.05, B))
        # drafts that are often what is sampled: each position's most likely token
        fed = torch.roll(s["logits"].float().argmax(-1).int(), 1, 1)
        s["fed"] = torch.where(uniform(0, 1, B, W) < 0.1, whole(0, V, B, W), fed).contiguous()
        s["tokens"] = torch.empty(B, W, dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty(B, W, device="cuda")
        s["n_reject"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s

    B, H, G, P, N = (case[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    io = _io(case)
    # step sizes between 0.001 and 0.1 at a zero projection, decay rates between 1 and 16
    dt0 = torch.exp(uniform(math.log(1e-3), math.log(0.1), H))
    dt_bias = dt0 + torch.log(-torch.expm1(-dt0))
    a_log = torch.log(uniform(1, 16, H))
    s["err"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    if case["op"] == "scan":
        T = case["tokens"]
        act = torch.nn.functional.silu
        s["cu"] = _cu(case)
        s["q"], s["k"] = (act(normal(T, G, N)).to(io) for _ in range(2))
        s["v"] = act(normal(T, H, P)).to(io)
        s["dt"] = torch.nn.functional.softplus(normal(T, H) + dt_bias)
        s["a"] = torch.exp(-torch.exp(a_log) * s["dt"])
        s["s_in"] = normal(B, H, P, N) * 0.3 if case["resume"] else None
        s["y"] = torch.empty(T, H, P, dtype=io, device="cuda")
        s["s_out"] = torch.empty(B, H, P, N, device="cuda")
        return s

    C = _channels(case)
    s["weight"] = uniform(-0.5, 0.5, C, WIDTH)
    s["bias"] = uniform(-0.5, 0.5, C)
    s["dt_bias"], s["a_log"] = dt_bias, a_log
    if case["op"] == "conv_prompt":
        rows, slots = case["tokens"], WIDTH - 1
        s["cu"] = _cu(case)
        s["state_in"] = normal(B, slots, C).to(io) if case["resume"] else None
        s["state_out"] = torch.empty(B, slots, C, dtype=io, device="cuda")
        lead = (rows,)
    else:
        W = case["window"]
        rows, slots = B * W, WIDTH - 1 + W
        s["state"] = normal(B, slots, C).to(io)
        s["pos"] = whole(8, 5000, B)
        s["base"] = s["pos"] - whole(0, 8, B)
        s["n_reject"] = torch.minimum(whole(0, W, B), s["pos"] - s["base"]) if case["rollback"] else None
        lead = (B, W)
    # the layer's projection: [gate | v, k, q before the convolution | dt before its softplus]
    s["rows"] = normal(rows, H * P + C + H).to(io)
    s["x"], s["dt_raw"] = s["rows"][:, H * P:H * P + C], s["rows"][:, H * P + C:]
    s["q"], s["k"] = (torch.empty(*lead, G, N, dtype=io, device="cuda") for _ in range(2))
    s["v"] = torch.empty(*lead, H, P, dtype=io, device="cuda")
    s["dt"], s["a"] = (torch.empty(*lead, H, device="cuda") for _ in range(2))
    return s


# ---- the plain forms -------------------------------------------------------

def _padded(cu, most):
    """Row of each (sequence, token) in the packed order, and whether there is one."""
    at = torch.arange(most, device=cu.device)
    there = at < (cu[1:] - cu[:-1]).unsqueeze(1)
    return torch.where(there, cu[:-1].unsqueeze(1) + at, 0).long(), there


def _plain_scan(s):
    c = s["case"]
    B, H, G, P, N = (c[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    Q, R = CHUNK, H // G
    nc = -(-max(lengths(c)) // Q)
    row, there = _padded(s["cu"], nc * Q)

    def chunks(t, heads, width):   # [B, nc, heads, Q, width]
        return t.float()[row].view(B, nc, Q, heads, width).transpose(2, 3)

    q, k, v = chunks(s["q"], G, N), chunks(s["k"], G, N), chunks(s["v"], H, P)
    dt = torch.where(there.unsqueeze(-1), s["dt"][row], 0).view(B, nc, Q, H).transpose(2, 3)
    a = torch.where(there.unsqueeze(-1), s["a"][row], 1).view(B, nc, Q, H).transpose(2, 3)
    csum = torch.cumsum(torch.log(a.double()), -1)                      # [B, nc, H, Q]
    lower = torch.ones(Q, Q, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp(torch.where(lower, (csum.unsqueeze(-1) - csum.unsqueeze(-2)), -math.inf).float())
    score = (q @ k.transpose(-1, -2)).repeat_interleave(R, 2)            # [B, nc, H, Q, Q]
    y = (score * decay * dt.unsqueeze(-2)) @ v
    last = torch.exp((csum[..., -1:] - csum).float()) * dt
    local = (v * last.unsqueeze(-1)).transpose(-1, -2) @ k.repeat_interleave(R, 2)     # [B, nc, H, P, N]
    # the state before chunk c: every earlier chunk's part, decayed from its end; row nc is the last state
    total = torch.cumsum(csum[..., -1], 1).transpose(1, 2)               # [B, H, nc]
    before = torch.nn.functional.pad(total, (1, 0))
    earlier = torch.ones(nc + 1, nc, dtype=torch.bool, device=q.device).tril(-1)
    carry = torch.exp(torch.where(earlier, before.unsqueeze(-1) - total.unsqueeze(-2), -math.inf).float())
    state = (carry @ local.transpose(1, 2).reshape(B, H, nc, P * N)).view(B, H, nc + 1, P, N)
    if s["s_in"] is not None:
        state = state + torch.exp(before.float())[..., None, None] * s["s_in"].unsqueeze(2)
    start = state[:, :, :nc].transpose(1, 2)
    y = y + torch.exp(csum.float()).unsqueeze(-1) * (q.repeat_interleave(R, 2) @ start.transpose(-1, -2))
    y = y.transpose(2, 3).reshape(B, nc * Q, H, P)[there]
    return {"y": y.to(s["y"].dtype), "s_out": state[:, :, nc].contiguous()}


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _inputs(s, x, raw, lead):
    """v, k, q, dt, a from the convolution's sums and the raw step sizes."""
    c = s["case"]
    H, G, P, N = (c[n] for n in ("heads", "groups", "head_dim", "state_dim"))
    io = s["q"].dtype
    o = _silu(x + s["bias"]).to(io).view(*lead, -1)
    dt = _softplus(raw.float() + s["dt_bias"]).view(*lead, H)
    v, k, q = torch.split(o, [H * P, G * N, G * N], -1)
    return {"v": v.reshape(*lead, H, P), "k": k.reshape(*lead, G, N), "q": q.reshape(*lead, G, N),
            "dt": dt, "a": torch.exp(-torch.exp(s["a_log"]) * dt)}


def _plain_conv_prompt(s):
    c = s["case"]
    B, T, K = c["batch"], c["tokens"], WIDTH
    cu = s["cu"].long()
    old = s["state_in"] if s["state_in"] is not None else torch.zeros_like(s["state_out"])
    # each sequence's rows behind its history: token i of sequence b at row cu[b] + b (K-1) + K-1 + i
    flat = torch.zeros(T + B * (K - 1), s["x"].shape[1], device=cu.device)
    seq = torch.repeat_interleave(torch.arange(B, device=cu.device), cu[1:] - cu[:-1], output_size=T)
    at = torch.arange(T, device=cu.device) + (seq + 1) * (K - 1)
    lead = (cu[:-1] + torch.arange(B, device=cu.device) * (K - 1)).unsqueeze(1) + torch.arange(K - 1, device=cu.device)
    flat[at] = s["x"].float()
    flat[lead] = old.float()
    taps = torch.stack([flat[at - (K - 1) + j] * s["weight"][:, j] for j in range(K)])
    tail = (cu[1:] + torch.arange(1, B + 1, device=cu.device) * (K - 1)).unsqueeze(1) - torch.arange(K - 1, 0, -1, device=cu.device)
    return {**_inputs(s, taps.sum(0), s["dt_raw"], (T,)), "state": flat[tail].to(s["q"].dtype)}


def _plain_conv_step(s):
    c = s["case"]
    B, W, K = c["batch"], c["window"], WIDTH
    R = s["state"].shape[1]
    pos = s["pos"].long()
    if s["n_reject"] is not None:
        drop = s["n_reject"].long()
        pos = torch.where((drop >= 0) & (drop <= pos - s["base"]), pos - drop, pos)
    seq = torch.arange(B, device=pos.device).unsqueeze(1)
    behind = (pos.unsqueeze(1) + torch.arange(1 - K, 0, device=pos.device)) % R
    x = s["x"].reshape(B, W, -1)
    rows = torch.cat([s["state"][seq, behind], x], 1).float()            # [B, K-1+W, C]
    taps = torch.stack([rows[:, j:j + W] * s["weight"][:, j] for j in range(K)])
    state = s["state"].clone()
    state[seq, (pos.unsqueeze(1) + torch.arange(W, device=pos.device)) % R] = x
    return {**_inputs(s, taps.sum(0), s["dt_raw"], (B, W)), "state": state}


def _plain_sample(s):
    x = s["logits"].double()
    B, W, V = x.shape

    def each(name, off):   # a sequence's setting, for each of its positions
        t = s.get(name)
        return torch.full((B, 1, 1), off, device=x.device) if t is None else t.view(B, 1, 1)

    temperature = each("temperature", 1.0).double()
    value, order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    scaled = (value.double() - x.amax(-1, keepdim=True)) / torch.where(temperature > 0, temperature, 1.0)
    weight = torch.round(torch.exp(scaled) * ONE).long()
    rank = torch.arange(V, device=x.device)
    top_k = each("top_k", 0)
    keep = (rank < top_k) | (top_k <= 0)
    weight = torch.where(keep, weight, 0)
    upto = torch.cumsum(weight, -1)
    top_p = each("top_p", 1.0).double()
    least = torch.ceil(top_p * upto[..., -1:].double()).long()
    keep = keep & ((upto - weight < least) | (top_p >= 1) | (rank == 0))
    keep = keep & (weight >= torch.ceil(each("min_p", 0.0).double() * ONE).long())
    kept = torch.zeros_like(weight).scatter_(-1, order, torch.where(keep, weight, 0))   # back in the vocabulary's order
    upto = torch.cumsum(kept, -1)
    mass = upto[..., -1]
    at = torch.minimum(torch.floor(s["u"].double() * mass.double()).long(), mass - 1)
    token = (upto <= at.unsqueeze(-1)).sum(-1)
    share = kept.gather(-1, token.unsqueeze(-1)).squeeze(-1).double() / mass.double()
    greedy = temperature.squeeze(-1) <= 0
    token = torch.where(greedy, order[..., 0], token).int()
    match = torch.cumprod((token[:, :-1] == s["fed"][:, 1:]).int(), 1)
    return {"tokens": token, "probs": torch.where(greedy, 1.0, share).float(), "n_reject": (W - 1 - match.sum(1)).int()}


# ---- the library's calls ---------------------------------------------------

def _kept(s):
    """What a serving program keeps from call to call: the layer's shape, its convolution, a workspace."""
    import linear_attention_decode_amd as lad
    if "kept" not in s:
        c, kept = s["case"], {}
        if c["op"] == "sample":
            need = lad.replay_sample_workspace(c["batch"], c["window"], c["vocab"])
        else:
            kept["cfg"] = lad.ReplayConfig(c["batch"], c["heads"], c["groups"], c["head_dim"], c["state_dim"], 16,
                                           lad.BF16 if c["io"] == "bf16" else lad.F32, lad.NONE, 0)
            need = 0
            if c["op"] == "scan":
                kept["most"] = max(lengths(c))
                need = lad.replay_scan_workspace(kept["cfg"], c["tokens"], kept["most"])
            else:
                slots = WIDTH - 1 + c.get("window", 0)
                kept["conv"] = lad.ReplayConv(s["weight"], s["bias"], s["dt_bias"], s["a_log"], slots=slots)
        kept["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        s["kept"] = kept
    return lad, s["kept"]


def _own(s):
    lad, kept = _kept(s)
    c = s["case"]
    if c["op"] == "scan":
        lad.replay_scan(kept["cfg"], c["tokens"], kept["most"], s["cu"], s["q"], s["k"], s["v"], s["dt"], s["a"], s["s_in"],
                        s["s_out"], s["y"], s["err"], kept["workspace"])
        return {"y": s["y"], "s_out": s["s_out"]}
    if c["op"] == "sample":
        lad.replay_sample(s["logits"], s["u"], s["tokens"], temperature=s.get("temperature"), top_k=s.get("top_k"),
                          top_p=s.get("top_p"), min_p=s.get("min_p"), probs=s["probs"], fed=s["fed"],
                          n_reject=s["n_reject"], workspace=kept["workspace"])
        return {n: s[n] for n in ("tokens", "probs", "n_reject")}
    outs = (s["q"], s["k"], s["v"], s["dt"], s["a"])
    if c["op"] == "conv_prompt":
        lad.replay_conv_prompt(kept["cfg"], kept["conv"], c["tokens"], s["cu"], s["x"], s["dt_raw"], None, s["state_in"],
                               s["state_out"], *outs, s["err"])
        state = s["state_out"]
    else:
        lad.replay_conv_step(kept["cfg"], kept["conv"], c["window"], s["x"], s["dt_raw"], s["pos"], s["state"], *outs,
                             base=s["base"], n_reject=s["n_reject"])
        state = s["state"]
    return {**{n: s[n] for n in ("q", "k", "v", "dt", "a")}, "state": state}


def run(state):
    if own:
        return _own(state)
    return {"scan": _plain_scan, "conv_prompt": _plain_conv_prompt, "conv_step": _plain_conv_step,
            "sample": _plain_sample}[state["case"]["op"]](state)


# ---- what a pass cannot do without, and what it should give ------------------

def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "sample":
        rows = case["batch"] * case["window"]
        # the logits once; a comparison, a difference, an exponential and a sum each
        return {"bytes": rows * (case["vocab"] * e + 16) + case["batch"] * 20, "flops": 4 * rows * case["vocab"]}
    B, H, G, P, N = (case[n] for n in ("batch", "heads", "groups", "head_dim", "state_dim"))
    if case["op"] == "scan":
        T = case["tokens"]
        states = B * H * P * N * 4 * (2 if case["resume"] else 1)
        # v, y, q, k, dt and a once, and the states; v k^T into the state and S q out of it
        return {"bytes": T * (2 * H * P * e + 2 * G * N * e + 8 * H) + states, "flops": 4 * T * H * P * N}
    C = _channels(case)
    if case["op"] == "conv_prompt":
        rows, states = case["tokens"], B * (WIDTH - 1) * C * e * (2 if case["resume"] else 1)
    else:
        rows, states = B * case["window"], B * (WIDTH - 1 + case["window"]) * C * e
    # rows in and out, dt and a; the taps and the activation
    return {"bytes": rows * (2 * C * e + H * (e + 8)) + states + C * (WIDTH + 1) * 4, "flops": rows * C * (2 * WIDTH + 4)}


def _exact_scan(case, s):
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
        k, q = (s[m][row].double().repeat_interleave(H // G, 1) for m in ("k", "q"))
        u = s["v"][row].double() * s["dt"][row].double().unsqueeze(-1)
        S[:n].mul_(s["a"][row].double()[..., None, None]).add_(u.unsqueeze(-1) * k.unsqueeze(-2))
        y[row] = (S[:n] * q.unsqueeze(-2)).sum(-1)
    out = torch.empty_like(S)
    out[by] = S
    return {"y": y, "s_out": out}


def _exact_conv(case, s):
    """Tap after tap in 64 bits, each row's history looked up by its place in the sequence."""
    H, G, P, N = (case[n] for n in ("heads", "groups", "head_dim", "state_dim"))
    B, K, C = case["batch"], WIDTH, _channels(case)
    x = s["x"].double()
    if case["op"] == "conv_prompt":
        lens = lengths(case)
        R = K - 1
        old, pos = s["state_in"], [0] * B
        state = torch.zeros(B, R, C, dtype=torch.float64, device="cuda")
        lead = (case["tokens"],)
    else:
        lens = [case["window"]] * B
        R = s["state"].shape[1]
        old, pos = s["state"], s["pos"].tolist()
        if s["n_reject"] is not None:
            pos = [p - r if 0 <= r <= p - b else p for p, r, b in zip(pos, s["n_reject"].tolist(), s["base"].tolist())]
        state = s["state"].double().clone()
        lead = (B, case["window"])
    sums = torch.empty_like(x)
    start = 0
    for b, n in enumerate(lens):
        behind = [(pos[b] - i) % R for i in range(K - 1, 0, -1)]
        hist = torch.zeros(K - 1, C, dtype=torch.float64, device="cuda") if old is None else old[b, behind].double()
        rows = torch.cat([hist, x[start:start + n]])
        acc = s["bias"].double().expand(n, C).clone()
        for j in range(K):
            acc += s["weight"][:, j].double() * rows[j:j + n]
        sums[start:start + n] = acc
        if case["op"] == "conv_prompt":
            for i in range(1, K):
                state[b, (pos[b] - i) % R] = rows[len(rows) - i]
        else:
            for i in range(n):
                state[b, (pos[b] + i) % R] = x[start + i]
        start += n
    o = sums * torch.sigmoid(sums)
    raw = s["dt_raw"].double() + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    a = torch.exp(-torch.exp(s["a_log"].double()) * dt)
    return {"v": o[:, :H * P].reshape(*lead, H, P), "k": o[:, H * P:H * P + G * N].reshape(*lead, G, N),
            "q": o[:, H * P + G * N:].reshape(*lead, G, N), "dt": dt.reshape(*lead, H), "a": a.reshape(*lead, H), "state": state}


def _exact_sample(case, s):
    """The chosen tokens' shares, row by row on the host in 64-bit floating point."""
    def each(name, off):
        return s[name].double().cpu().numpy() if name in s else np.full(case["batch"], off)

    temperature, top_k, top_p, min_p = each("temperature", 1.0), each("top_k", 0), each("top_p", 1.0), each("min_p", 0.0)
    share = np.ones((case["batch"], case["window"]))
    for b in range(case["batch"]):
        if temperature[b] <= 0:
            continue
        for w, x in enumerate(s["logits"][b].double().cpu().numpy()):
            order = np.argsort(-x, kind="stable")
            if top_k[b] > 0:
                order = order[:int(top_k[b])]
            p = np.exp((x[order] - x[order[0]]) / temperature[b])
            stay = p >= min_p[b]
            if top_p[b] < 1:
                ahead = np.concatenate([[0.0], np.cumsum(p)[:-1]])
                stay &= (ahead < top_p[b] * p.sum()) | (np.arange(len(p)) == 0)
            by = np.argsort(order[stay])
            p = p[stay][by]
            upto = np.cumsum(p)
            at = min(np.searchsorted(upto, float(s["u"][b, w]) * upto[-1], side="right"), len(p) - 1)
            share[b, w] = p[at] / upto[-1]
    return {"tokens": None, "probs": torch.from_numpy(share), "n_reject": None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    return _exact_scan(case, s) if case["op"] == "scan" else _exact_conv(case, s)
