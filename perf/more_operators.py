"""The cases that the operators of a hybrid decoder layer beside its attention
are measured on, with their plain forms.

Three operators take a step's new tokens -- single ones, verify blocks, chunks
of prompts -- through such a layer:

  gdn_inputs    short convolution, SiLU, norms of the heads and gates: what the
                gated delta rule reads, from the layer's projections
  gdn_advance   the gated delta rule over packed rows, the states in place:
                token by token for a few rows, in chunks for a prompt
  moe_smallm    a whole mixture-of-experts layer for few rows: router, the
                chosen 4-bit experts' products, their weighted sum

Layouts: packed rows (the sequences' new tokens one after another, sequence b's
at q_start[b]:q_start[b + 1], zeros past the last), states fp32
[slots][heads][dv][dk], windows fp32 [slots][W - 1][channels], weights 4-bit
affine in groups of 64 (words of eight nibbles, bf16 scales and biases).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one request's verify block of K + 1 = 4 rows, fp32 to fp32 for the tape;
        # its window is committed later
        {"name": "inputs: one verify block", "op": "inputs", "seqs": 1, "new_lo": 4, "new_hi": 4,
         "kheads": 48, "heads": 48, "dk": 128, "dv": 128, "width": 4, "src": "f32", "dst": "f32",
         "update": False, "mix": 1},
        # a server's single tokens, shared key heads
        {"name": "inputs: 256 tokens", "op": "inputs", "seqs": 256, "new_lo": 1, "new_hi": 1,
         "kheads": 16, "heads": 48, "dk": 128, "dv": 128, "width": 4, "src": "bf16", "dst": "bf16",
         "update": True, "mix": 2},
        # chunks of three prompts
        {"name": "inputs: prompts", "op": "inputs", "seqs": 3, "new_lo": 1000, "new_hi": 4001,
         "kheads": 16, "heads": 48, "dk": 128, "dv": 128, "width": 4, "src": "bf16", "dst": "bf16",
         "update": True, "mix": 3},
        # a single token of one request: latency
        {"name": "advance: one token", "op": "advance", "seqs": 1, "new_lo": 1, "new_hi": 1,
         "kheads": 16, "heads": 48, "dk": 128, "dv": 128, "dtype": "bf16", "empty": False, "mix": 4},
        # single tokens of a batch: the states' traffic
        {"name": "advance: 64 tokens", "op": "advance", "seqs": 64, "new_lo": 1, "new_hi": 1,
         "kheads": 48, "heads": 48, "dk": 128, "dv": 128, "dtype": "bf16", "empty": False, "mix": 5},
        # a few fp32 rows each, narrow keys, a sequence without rows
        {"name": "advance: short ragged", "op": "advance", "seqs": 9, "new_lo": 1, "new_hi": 13,
         "kheads": 20, "heads": 20, "dk": 64, "dv": 128, "dtype": "f32", "empty": True, "mix": 6},
        # one whole prompt
        {"name": "advance: one prompt", "op": "advance", "seqs": 1, "new_lo": 5000, "new_hi": 5000,
         "kheads": 48, "heads": 48, "dk": 128, "dv": 128, "dtype": "bf16", "empty": False, "mix": 7},
        # prompts of different lengths, packed, shared key heads
        {"name": "advance: packed prompts", "op": "advance", "seqs": 5, "new_lo": 77,
         "new_hi": 2001, "kheads": 16, "heads": 48, "dk": 128, "dv": 128, "dtype": "bf16",
         "empty": False, "mix": 8},
        # one token, many small experts: latency
        {"name": "experts: one token", "op": "experts", "rows": 1, "hidden": 2048, "inter": 512,
         "experts": 256, "top": 8},
        # a verify block of a wide model
        {"name": "experts: verify block", "op": "experts", "rows": 4, "hidden": 5120,
         "inter": 1024, "experts": 64, "top": 6},
        # a few requests' tokens, sizes that no tile divides
        {"name": "experts: 19 tokens", "op": "experts", "rows": 19, "hidden": 2560, "inter": 896,
         "experts": 60, "top": 4},
        # 32 verify blocks
        {"name": "experts: 32 verify blocks", "op": "experts", "rows": 128, "hidden": 2048,
         "inter": 1024, "experts": 96, "top": 6},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["inputs", "advance", "advance", "advance", "experts", "experts"])
    if op == "experts":
        while True:
            hidden, inter = 128 * rng.randint(4, 40), 128 * rng.randint(1, 12)
            experts = _log(rng, 4, 256)
            if experts * hidden * inter <= 96 * 2048 * 1024:
                break
        return {"op": op, "rows": _log(rng, 1, 128), "hidden": hidden, "inter": inter,
                "experts": experts, "top": rng.randint(1, min(experts, 10))}
    kheads = rng.choice([1, 2, 4, 8, 16])
    heads = kheads * rng.choice([1, 1, 2, 3])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (96, 80)])
    kind = rng.choice(["token", "verify", "prompt", "prompt"])
    if kind == "prompt":
        seqs = rng.choice([1, 1, 2, 3, 6])
        new = _log(rng, 17, 5000)
        while seqs * new * heads > 240000:
            new = new * 3 // 4
        lo = max(1, new // 10)
    else:
        seqs = _log(rng, 1, 256 if op == "inputs" else 64)
        lo, new = (1, 1) if kind == "token" else (1, rng.choice([2, 4, 9, 16]))
    c = {"op": op, "seqs": seqs, "new_lo": lo, "new_hi": new, "kheads": kheads, "heads": heads,
         "dk": dk, "dv": dv, "mix": rng.randrange(1 << 20)}
    if op == "inputs":
        src = rng.choice(["bf16", "f32"])
        c.update(width=rng.choice([2, 4, 4, 5, 8]), src=src,
                 dst="bf16" if kind == "prompt" else rng.choice(["bf16", "f32"]),
                 update=rng.random() < 0.7)
    else:
        c.update(dtype="bf16" if kind == "prompt" else rng.choice(["bf16", "f32"]),
                 empty=seqs > 2 and rng.random() < 0.5)
    return c


PAD = 3  # rows past the last sequence: a captured step's padding


def _lengths(c):
    """Each sequence's new rows: a function of the case alone."""
    r = random.Random(c["mix"])
    new = [c["new_hi"] if c["new_lo"] == c["new_hi"] else _log(r, c["new_lo"], c["new_hi"])
           for _ in range(c["seqs"])]
    new[-1] = c["new_hi"]
    if c.get("empty"):
        new[1] = 0
    return new


def _channels(c):
    return 2 * c["kheads"] * c["dk"] + c["heads"] * c["dv"]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"inputs": _prepare_inputs, "advance": _prepare_advance,
            "experts": _prepare_experts}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _packed(c, g):
    """q_start, the slots of the sequences (of two more than there are), rows."""
    new = _lengths(c)
    start = [0]
    for t in new:
        start.append(start[-1] + t)
    slots = torch.randperm(c["seqs"] + 2, generator=g, device=DEV)[:c["seqs"]].to(torch.int32)
    return torch.tensor(start, dtype=torch.int32, device=DEV), slots, start[-1] + PAD


def _prepare_inputs(c, g):
    q_start, slots, rows = _packed(c, g)
    C, W, H = _channels(c), c["width"], c["heads"]
    dt, to = _type(c["src"]), _type(c["dst"])
    # the projections' outputs: the gates' columns are slices of one projection's rows
    gates = _randn(g, rows, 2 * H, dtype=dt)
    s = {"case": c, "q_start": q_start, "slots": slots, "rows": rows, "max_new": max(_lengths(c)),
         "x": _randn(g, rows, C, dtype=dt), "a": gates[:, :H], "b": gates[:, H:],
         "weight": _randn(g, W, C, std=1.0 / math.sqrt(W)),
         "window": _randn(g, c["seqs"] + 2, W - 1, C),
         "a_log": _randn(g, H).mul_(1.5).sub_(2.0), "dt_bias": _randn(g, H),
         "scale": 1.0 / math.sqrt(c["dk"])}
    s["out"] = (torch.zeros(rows, c["kheads"], c["dk"], dtype=to, device=DEV),
                torch.zeros(rows, c["kheads"], c["dk"], dtype=to, device=DEV),
                torch.zeros(rows, H, c["dv"], dtype=to, device=DEV),
                torch.zeros(rows, H, device=DEV), torch.zeros(rows, H, device=DEV))
    return s


def _prepare_advance(c, g):
    q_start, slots, rows = _packed(c, g)
    dt, H = _type(c["dtype"]), c["heads"]

    def unit(heads):
        x = _randn(g, rows, heads, c["dk"])
        return x / x.square().sum(-1, keepdim=True).sqrt()

    # heads forget at rates from a few tokens to thousands
    rate = torch.exp(_rand(g, H) * math.log(1e-3))
    decay = torch.exp(-rate * torch.log1p(torch.exp(_randn(g, rows, H))))
    return {"case": c, "q_start": q_start, "slots": slots, "rows": rows,
            "max_new": max(_lengths(c)), "q": (unit(c["kheads"]) / math.sqrt(c["dk"])).to(dt),
            "k": unit(c["kheads"]).to(dt), "v": _randn(g, rows, H, c["dv"], dtype=dt),
            "alpha": decay, "beta": torch.sigmoid(_randn(g, rows, H)),
            "state": _randn(g, c["seqs"] + 2, H, c["dv"], c["dk"], std=0.05),
            "out": torch.zeros(rows, H, c["dv"], dtype=dt, device=DEV)}


def _prepare_experts(c, g):
    H, I, E = c["hidden"], c["inter"], c["experts"]

    def four_bit(n, k):
        """Weights of about N(0, 1 / k), in groups with scales of their own."""
        words = torch.randint(-2**31, 2**31, (E, n, k // 8), generator=g, device=DEV,
                              dtype=torch.int64).to(torch.int32)
        scales = (_rand(g, E, n, k // 64) + 0.5).mul_(1 / (4.6 * math.sqrt(k)))
        return words, scales.bfloat16(), (scales * -7.5).bfloat16()

    s = {"case": c, "x": _randn(g, c["rows"], H, dtype=torch.bfloat16),
         "router": _randn(g, E, H, std=1.0 / math.sqrt(H)).bfloat16(),
         "gate": four_bit(I, H), "up": four_bit(I, H), "down": four_bit(H, I),
         "out": torch.zeros(c["rows"], H, dtype=torch.bfloat16, device=DEV)}
    if own:
        import mtp_speculative_decoding_qmv_gb300 as sv

        s["workspace"] = sv.make_moe_workspace(c["rows"], H, I, E, c["top"], torch.device(DEV, 0))
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    if own:
        return {"inputs": _own_inputs, "advance": _own_advance,
                "experts": _own_experts}[s["case"]["op"]](s)
    return {"inputs": _plain_inputs, "advance": _plain_advance,
            "experts": _plain_experts}[s["case"]["op"]](s)


def _own_inputs(s):
    import mtp_speculative_decoding_qmv_gb300 as sv

    sv.gdn_inputs(s["x"], s["a"], s["b"], s["weight"], s["window"], s["a_log"], s["dt_bias"],
                  s["q_start"], s["max_new"], window_index=s["slots"],
                  update_window=s["case"]["update"], q_scale=s["scale"], out=s["out"])
    return (*s["out"], s["window"])


def _own_advance(s):
    import mtp_speculative_decoding_qmv_gb300 as sv

    sv.gdn_advance(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["state"], s["q_start"],
                   s["max_new"], state_index=s["slots"], out=s["out"])
    return s["out"], s["state"]


def _own_experts(s):
    import mtp_speculative_decoding_qmv_gb300 as sv

    return sv.moe_smallm(s["x"], s["router"], s["gate"], s["up"], s["down"], s["case"]["top"],
                         out=s["out"], workspace=s["workspace"])


def _places(s):
    """For every row its sequence, its place in it and whether it belongs to one."""
    start = s["q_start"].long()
    r = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), r, right=True)
    real = b < s["case"]["seqs"]
    b = b.clamp(max=s["case"]["seqs"] - 1)
    return b, r - start[b], real


def _plain_inputs(s):
    c = s["case"]
    W, Hk, H, rows = c["width"], c["kheads"], c["heads"], s["rows"]
    b, t, real = _places(s)
    x, window, slot = s["x"].float(), s["window"], s["slots"].long()
    tap = torch.arange(W, device=DEV)
    at = t[:, None] - (W - 1) + tap  # the taps' places in the sequence; before 0: the window's
    r = torch.arange(rows, device=DEV)[:, None] - (W - 1) + tap
    h = torch.where((at >= 0)[..., None], x[r.clamp(min=0)],
                    window[slot[b][:, None], (at + W - 1).clamp(max=W - 2)])
    y = (h * s["weight"]).sum(1)
    y = y * torch.sigmoid(y)
    q, k, v = y.split([Hk * c["dk"], Hk * c["dk"], H * c["dv"]], 1)

    def unit(z):
        z = z.view(rows, Hk, c["dk"])
        return z * torch.rsqrt(z.square().sum(-1, keepdim=True) + 1e-6)

    z = s["a"].float() + s["dt_bias"]
    softplus = torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
    alpha = torch.exp(-torch.exp(s["a_log"]) * softplus)
    keep = real[:, None]
    for to, val in zip(s["out"], (unit(q) * s["scale"], unit(k), v.reshape(rows, H, c["dv"]),
                                  alpha, torch.sigmoid(s["b"].float()))):
        to.copy_(torch.where(keep if val.dim() == 2 else keep[..., None], val, 0.0))
    if c["update"]:
        start = s["q_start"].long()
        n = start[1:] - start[:-1]
        last = n[:, None] - (W - 1) + tap[:-1]  # the places whose inputs the window holds next
        row = (start[:-1, None] + last).clamp(0, rows - 1)
        window[slot] = torch.where((last >= 0)[..., None], x[row],
                                   window[slot[:, None], (last + W - 1).clamp(max=W - 2)])
    return (*s["out"], window)


def _plain_advance(s):
    """In chunks of C rows: with D[i][j] the gates' product from j + 1 to i and
    G[i] that from the chunk's first to i, the rows e solve
    (1 + tril(beta K K' D, -1)) e = beta (v - G K S'), o = G Q S' + tril(Q K' D) e,
    and the next state is G[last] S + e' D[last] K."""
    c = s["case"]
    B, H, dk, dv = c["seqs"], c["heads"], c["dk"], c["dv"]
    C = min(64, s["max_new"])
    N = -(-s["max_new"] // C)
    start = s["q_start"].long()
    n = (start[1:] - start[:-1])[:, None]
    t = torch.arange(N * C, device=DEV)
    real = t < n
    row = (start[:-1, None] + t).clamp(max=s["rows"] - 1)

    def chunks(x, fill=0.0):  # [B, H, N, C, width or none]
        x = x.float()
        if x.dim() == 3 and x.shape[1] != H:
            x = x.repeat_interleave(H // x.shape[1], 1)
        x = x[row]
        x = torch.where(real.view(B, -1, *[1] * (x.dim() - 2)), x, fill)
        return x.view(B, N, C, *x.shape[2:]).movedim(3, 1)

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    beta = chunks(s["beta"])[..., None]
    G = chunks(s["alpha"], 1.0).double().log().cumsum(-1)
    i = torch.arange(C, device=DEV)
    lower = i[:, None] >= i
    D = torch.where(lower, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    P = q @ k.transpose(-1, -2) * D
    L = torch.where(i[:, None] > i, beta * (k @ k.transpose(-1, -2)) * D, 0.0)
    G = G.exp().float()[..., None]
    T = torch.eye(C, device=DEV).expand_as(L).contiguous()
    for m in range(1, C):
        T[..., m, :m] = -(L[..., m:m + 1, :m] @ T[..., :m, :m]).squeeze(-2)
    W, U = T @ (beta * G * k), T @ (beta * v)
    k, q, slot = k * D[..., -1, :, None], q * G, s["slots"].long()
    S = s["state"][slot].transpose(-1, -2)
    o = torch.empty(B, H, N, C, dv, device=DEV)
    for m in range(N):
        e = U[:, :, m] - W[:, :, m] @ S
        o[:, :, m] = q[:, :, m] @ S + P[:, :, m] @ e
        S = S * G[:, :, m, -1:] + k[:, :, m].transpose(-1, -2) @ e
    s["state"][slot] = S.transpose(-1, -2)
    b, at, mine = _places(s)
    o = o.view(B, H, N * C, dv)[b, :, at.clamp(max=N * C - 1)]
    s["out"].copy_(torch.where(mine[:, None, None], o, 0.0))
    return s["out"], s["state"]


def _plain_weights(w, ids=None):
    words, scales, biases = w if ids is None else (x[ids] for x in w)
    nibble = torch.arange(0, 32, 4, dtype=torch.int32, device=DEV)
    q = ((words[..., None] >> nibble) & 15).flatten(-2).float()
    q = q.unflatten(-1, (-1, 64))
    return (q * scales.float()[..., None] + biases.float()[..., None]).flatten(-2)


def _plain_experts(s):
    c = s["case"]
    E, top, rows = c["experts"], c["top"], c["rows"]
    x = s["x"].float()
    logits = x @ s["router"].float().T
    chosen, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    chosen, ids = chosen[:, :top], ids[:, :top]
    weight = (chosen - chosen[:, :1]).exp()
    weight = weight / weight.sum(-1, keepdim=True)
    if rows * top < E:  # the chosen experts' weights alone
        ids = ids.flatten()
        x = x.repeat_interleave(top, 0)[..., None]
        gate, up = _plain_weights(s["gate"], ids) @ x, _plain_weights(s["up"], ids) @ x
        y = _plain_weights(s["down"], ids) @ (gate * torch.sigmoid(gate) * up)
        y = (y.view(rows, top, -1) * weight[..., None]).sum(1)
    else:  # every expert for every row, with a weight of 0 where it is not chosen
        all_weights = torch.zeros(rows, E, device=DEV).scatter_(1, ids, weight)
        gate = x @ _plain_weights(s["gate"]).transpose(1, 2)
        up = x @ _plain_weights(s["up"]).transpose(1, 2)
        y = (gate * torch.sigmoid(gate) * up) @ _plain_weights(s["down"]).transpose(1, 2)
        y = (y * all_weights.T[..., None]).sum(0)
    s["out"].copy_(y)
    return s["out"]


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "experts":
        T, H, I, E, k = c["rows"], c["hidden"], c["inter"], c["experts"], c["top"]
        met = E * (1.0 - (1.0 - k / E) ** T)  # experts that some row chooses, on average
        return {"bytes": met * 3 * H * I * 0.5625 + 2.0 * E * H + 4.0 * T * H,
                "flops": 6.0 * T * k * H * I + 2.0 * T * E * H}
    new = _lengths(c)
    rows = sum(new) + PAD
    if c["op"] == "inputs":
        C, H, W = _channels(c), c["heads"], c["width"]
        size, to = (4 if c[x] == "f32" else 2 for x in ("src", "dst"))
        window = c["seqs"] * (W - 1) * C * 4.0 * (2 if c["update"] else 1)
        return {"bytes": rows * (C * (size + to) + H * (2.0 * size + 8)) + window + W * C * 4.0,
                "flops": rows * C * (2.0 * W + 6)}
    size = 4 if c["dtype"] == "f32" else 2
    H, dk, dv = c["heads"], c["dk"], c["dv"]
    row = size * (2 * c["kheads"] * dk + 2 * H * dv) + 8 * H
    return {"bytes": float(rows * row + 8 * sum(n > 0 for n in new) * H * dk * dv),
            "flops": 6.0 * sum(new) * H * dk * dv}


# ----------------------------------------------------------------------------
# the definitions, in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"inputs": _exact_inputs, "advance": _exact_advance,
            "experts": _exact_experts}[case["op"]](case, s)


def _exact_inputs(c, s):
    W, Hk, dk = c["width"], c["kheads"], c["dk"]
    new = _lengths(c)
    out = [torch.zeros(o.shape, dtype=torch.float64, device=DEV) for o in s["out"]]
    window, row = s["window"].double(), 0
    a, beta = s["a"].double(), s["b"].double()
    for n, slot in zip(new, s["slots"].tolist()):
        if n == 0:
            continue
        past = torch.cat([window[slot], s["x"][row:row + n].double()])
        y = sum(past[j:j + n] * s["weight"][j].double() for j in range(W))
        y = y / (1 + torch.exp(-y))
        at = slice(row, row + n)
        for i in range(2):
            z = y[:, i * Hk * dk:(i + 1) * Hk * dk].reshape(n, Hk, dk)
            out[i][at] = z / ((z * z).sum(-1, keepdim=True) + 1e-6).sqrt()
        out[0][at] *= s["scale"]
        out[2][at] = y[:, 2 * Hk * dk:].reshape(n, c["heads"], c["dv"])
        soft = torch.logaddexp(a[at] + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device=DEV))
        out[3][at] = torch.exp(-soft * torch.exp(s["a_log"].double()))
        out[4][at] = 1 / (1 + torch.exp(-beta[at]))
        if c["update"]:
            window[slot] = past[n:]
        row += n
    return (*out, window)


def _exact_advance(c, s):
    """Token by token, the sequences side by side, the longest first."""
    new = _lengths(c)
    order = sorted(range(c["seqs"]), key=lambda b: -new[b])
    start = s["q_start"].tolist()
    G = c["heads"] // c["kheads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    state = s["state"].double()
    slot = s["slots"].long()[torch.tensor(order, device=DEV)]
    S = state[slot]
    alpha, beta = s["alpha"].double(), s["beta"].double()
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if G > 1:
        q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    for t in range(max(new)):
        live = sum(n > t for n in new)
        r = torch.tensor([start[b] + t for b in order[:live]], device=DEV)
        A = S[:live].mul_(alpha[r][:, :, None, None])
        e = beta[r][..., None] * (v[r] - torch.einsum("bhij,bhj->bhi", A, k[r]))
        A += e[..., None] * k[r][:, :, None]
        out[r] = torch.einsum("bhij,bhj->bhi", A, q[r])
    state[slot] = S
    return out, state


def _exact_experts(c, s):
    x = s["x"].double()
    logits = x @ s["router"].double().T
    y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    ranked = [sorted(range(c["experts"]), key=lambda e, z=z: (-z[e], e))[:c["top"]]
              for z in logits.tolist()]

    def matrix(w, e):
        words = w[0][e].to(torch.int64) & 0xFFFFFFFF
        q = torch.stack([(words >> (4 * i)) % 16 for i in range(8)], -1).reshape(words.shape[0], -1)
        return q.double() * w[1][e].double().repeat_interleave(64, 1) \
            + w[2][e].double().repeat_interleave(64, 1)

    for e in range(c["experts"]):
        mine = [t for t, best in enumerate(ranked) if e in best]
        if not mine:
            continue
        r = torch.tensor(mine, device=DEV)
        best = torch.tensor([ranked[t] for t in mine], device=DEV)
        share = 1 / torch.exp(logits[r[:, None], best] - logits[r, e][:, None]).sum(-1)
        g, u = x[r] @ matrix(s["gate"], e).T, x[r] @ matrix(s["up"], e).T
        y[r] += share[:, None] * ((g / (1 + torch.exp(-g)) * u) @ matrix(s["down"], e).T)
    return y
