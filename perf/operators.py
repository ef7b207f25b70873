"""The cases that the paged-cache operators are measured on, with their plain forms.

Three operators serve the attention layers beside the verify-and-accept path:

  kv_pages_step    pages, slots and positions of a step's new tokens, from the
                   requests' lengths
  rope_kv_append   rotary positions (and the norm of each head) for a step's
                   queries and keys, and the keys and values into their slots
  paged_attention  a step's new tokens -- one, a verify block, or a chunk of a
                   prompt -- over the paged cache

Layouts: caches bf16 [pages][kv heads][page size][head dim], block tables int32
[requests][most pages], packed rows (the requests' new tokens one after another,
request b's at q_start[b]:q_start[b + 1]).
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
        # one request's verify block of K + 1 = 4 rows: the latency of a cycle
        {"name": "pages, one verify block", "op": "pages", "requests": 1, "page": 16,
         "ctx_lo": 4093, "ctx_hi": 4093, "new_lo": 4, "new_hi": 4, "ended": 0, "mix": 1},
        # the verify blocks of a batch of 32
        {"name": "pages, 32 verify blocks", "op": "pages", "requests": 32, "page": 64,
         "ctx_lo": 100, "ctx_hi": 20000, "new_lo": 4, "new_hi": 4, "ended": 0, "mix": 2},
        # a large server's step: single tokens and prompt chunks together, some requests ending
        {"name": "pages, 1000 mixed requests", "op": "pages", "requests": 1000, "page": 16,
         "ctx_lo": 1, "ctx_hi": 30000, "new_lo": 1, "new_hi": 700, "ended": 37, "mix": 3},
        # the verify block of one request, straight from the 4-bit projections (fp32)
        {"name": "append, one verify block", "op": "append", "rows": 4, "heads": 40, "kv": 40,
         "dim": 128, "rot": 128, "axes": 1, "norm": False, "pairs": False, "dtype": "f32",
         "page": 16, "far": 30000},
        # 32 verify blocks of a model with images: three axes, normed heads, shared kv heads
        {"name": "append, 32 verify blocks", "op": "append", "rows": 128, "heads": 40, "kv": 8,
         "dim": 128, "rot": 128, "axes": 3, "norm": True, "pairs": False, "dtype": "bf16",
         "page": 64, "far": 200000},
        # a prompt chunk of a model with wide heads, a quarter of each rotated
        {"name": "append, prompt chunk", "op": "append", "rows": 8191, "heads": 20, "kv": 4,
         "dim": 256, "rot": 64, "axes": 1, "norm": True, "pairs": False, "dtype": "bf16",
         "page": 128, "far": 1000000},
        # a single token of one request over a short context: latency
        {"name": "attend, one token", "op": "attend", "requests": 1, "heads": 40, "kv": 8,
         "dim": 128, "page": 16, "ctx_lo": 999, "ctx_hi": 999, "new_lo": 1, "new_hi": 1,
         "window": 0, "empty": False, "mix": 1},
        # one request's verify block over a long context, a kv head for every head
        {"name": "attend, long verify", "op": "attend", "requests": 1, "heads": 40, "kv": 40,
         "dim": 128, "page": 64, "ctx_lo": 100001, "ctx_hi": 100001, "new_lo": 4, "new_hi": 4,
         "window": 0, "empty": False, "mix": 2},
        # a batch of verify blocks over ragged contexts
        {"name": "attend, 32 verify blocks", "op": "attend", "requests": 32, "heads": 40, "kv": 8,
         "dim": 128, "page": 64, "ctx_lo": 200, "ctx_hi": 30000, "new_lo": 4, "new_hi": 4,
         "window": 0, "empty": False, "mix": 3},
        # single tokens of a batch, wide heads, small pages
        {"name": "attend, 16 tokens, wide", "op": "attend", "requests": 16, "heads": 20, "kv": 4,
         "dim": 256, "page": 16, "ctx_lo": 1000, "ctx_hi": 20000, "new_lo": 1, "new_hi": 1,
         "window": 0, "empty": False, "mix": 4},
        # a whole prompt, causal
        {"name": "attend, whole prompt", "op": "attend", "requests": 1, "heads": 40, "kv": 8,
         "dim": 128, "page": 128, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 5000, "new_hi": 5000,
         "window": 0, "empty": False, "mix": 5},
        # prompt chunks of different lengths, packed, over what came before them
        {"name": "attend, packed chunks", "op": "attend", "requests": 3, "heads": 40, "kv": 8,
         "dim": 128, "page": 16, "ctx_lo": 3000, "ctx_hi": 30000, "new_lo": 77, "new_hi": 1000,
         "window": 0, "empty": False, "mix": 6},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["pages", "append", "append", "attend", "attend", "attend"])
    if op == "pages":
        B = _log(rng, 1, 1000)
        new = rng.choice([(1, 1), (1, 9), (4, 4), (1, 700)])
        return {"op": op, "requests": B, "page": rng.choice([16, 32, 64, 128]), "ctx_lo": 1,
                "ctx_hi": _log(rng, 10, 30000), "new_lo": new[0], "new_hi": new[1],
                "ended": rng.randint(0, B // 4), "mix": rng.randrange(1 << 20)}
    dim = rng.choice([64, 128, 128, 256])
    if op == "append":
        kv = rng.choice([1, 2, 4, 8, 16])
        return {"op": op, "rows": _log(rng, 1, 5000), "heads": kv * rng.choice([1, 2, 3, 5, 8]) if kv < 8
                else kv * rng.choice([1, 2, 3]), "kv": kv, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4]), "axes": rng.choice([1, 1, 3]),
                "norm": rng.random() < 0.5, "pairs": rng.random() < 0.3,
                "dtype": rng.choice(["bf16", "f32"]), "page": rng.choice([16, 32, 64, 128]),
                "far": _log(rng, 1000, 1000000)}
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 5, 8])
    kind = rng.choice(["token", "verify", "chunk", "chunk"])
    if kind == "chunk":
        # the plain form holds every score: requests x rows x heads x positions of them
        B = rng.choice([1, 1, 2, 3, 5])
        new = _log(rng, 20, 3000)
        ctx = _log(rng, 1, 20000)
        while B * new * heads * (ctx + new) > 1.0e9:
            new, ctx = max(1, new * 3 // 4), max(1, ctx * 3 // 4)
        lo = max(1, new // 8)
    else:
        B = _log(rng, 1, 64)
        new, lo = (1, 1) if kind == "token" else (rng.choice([2, 4, 5, 9]), 1)
        ctx = _log(rng, 10, 30000)
        while B * new * heads * (ctx + new) > 1.0e9 or B * (ctx + new) * kv * dim > 1.2e9:
            ctx = max(1, ctx * 3 // 4)
    return {"op": op, "requests": B, "heads": heads, "kv": kv, "dim": dim,
            "page": rng.choice([16, 32, 64, 128]), "ctx_lo": max(1, ctx // 30), "ctx_hi": ctx,
            "new_lo": lo, "new_hi": new, "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
            "empty": B > 2 and rng.random() < 0.5, "mix": rng.randrange(1 << 20)}


def _lengths(c):
    """Each request's committed length and new tokens: a function of the case alone."""
    r = random.Random(c["mix"])

    def some(lo, hi):
        return hi if lo == hi else _log(r, lo, hi)

    ctx = [some(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["requests"])]
    new = [some(c["new_lo"], c["new_hi"]) for _ in range(c["requests"])]
    if c["requests"] > 1:  # the ends of the ranges are always met
        ctx[0], new[-1] = c["ctx_hi"], c["new_hi"]
    return ctx, new


def _pages_of(tokens, page):
    return -(-tokens // page)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"pages": _prepare_pages, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _step_lengths(c):
    """For kv_pages_step: lengths before the previous step's commit, the commit,
    and the new tokens, with the ended requests' at -1."""
    ctx, new = _lengths(c)
    r = random.Random(c["mix"] + 1)
    commit = [r.randint(0, min(3, n - 1)) if n > 0 else 0 for n in ctx]
    for b in r.sample(range(c["requests"]), c["ended"]):
        new[b] = -1
    return ctx, commit, new


def _prepare_pages(c, g):
    ctx, commit, new = _step_lengths(c)
    page, B = c["page"], c["requests"]
    held = [_pages_of(n, page) for n in ctx]
    need = sum(max(0, _pages_of(n + t, page) - h) for n, t, h in zip(ctx, new, held) if t > 0)
    most = _pages_of(max(ctx) + max(new) + 8, page)
    total = sum(held) + need + 64
    ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, most, dtype=torch.int32, device=DEV)
    h = _ints(held)
    start = torch.cumsum(h, 0) - h
    at = torch.arange(most, device=DEV)[None, :]
    table = torch.where(at < h[:, None], ids[(start[:, None] + at).clamp(max=total - 1)], table)
    ring = torch.full((total,), -1, dtype=torch.int32, device=DEV)
    n_free = total - sum(held)
    head = int(torch.randint(0, total, (1,), generator=g, device=DEV))
    ring[(head + torch.arange(n_free, device=DEV)) % total] = ids[sum(held):]
    rows = sum(t for t in new if t > 0) + 5  # a captured step's rows: some of them padding
    s = {"case": c, "rows": rows, "page": page, "table": table.contiguous(), "ring": ring,
         "length": _ints([n - k - 1 for n, k in zip(ctx, commit)]), "held": h, "n_new": _ints(new),
         "commit": _ints(commit), "cursor": _ints([head, n_free]),
         "length_out": _ints([0] * B), "held_out": _ints([0] * B), "cursor_out": _ints([0, 0]),
         "q_start": _ints([0] * (B + 1)), "kv_len": _ints([0] * B), "slots": _ints([0] * rows),
         "positions": _ints([0] * rows), "flags": _ints([0] * B)}
    return s


def _inv_freq(c):
    half = c["rot"] // 2
    return torch.arange(half, dtype=torch.float64, device=DEV).mul_(-2.0 / c["rot"]).mul_(math.log(1e6)).exp_()


def _axis(c):
    """Which of the axes each rotary frequency turns by: three blocks, the first the widest."""
    half = c["rot"] // 2
    a, b = half // 2, half // 4
    return torch.tensor([0] * a + [1] * b + [2] * (half - a - b), dtype=torch.uint8, device=DEV)


def _prepare_append(c, g):
    rows, D, page = c["rows"], c["dim"], c["page"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    # one projection's output: the three are slices of its rows
    qkv = _randn(g, rows, c["heads"] + 2 * c["kv"], D, dtype=dt)
    pages = _pages_of(rows, page) + 3
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:rows].to(torch.int32)
    if rows > 8:
        slots[-3:] = -1  # padding rows
    pos = torch.randint(0, c["far"], (rows, c["axes"]), generator=g, device=DEV, dtype=torch.int32)
    s = {"case": c, "q": qkv[:, :c["heads"]], "k": qkv[:, c["heads"]:c["heads"] + c["kv"]],
         "v": qkv[:, c["heads"] + c["kv"]:], "positions": pos, "slots": slots,
         "inv_freq": _inv_freq(c), "axis": _axis(c) if c["axes"] > 1 else None,
         "q_weight": _randn(g, D).mul_(0.1).add_(1) if c["norm"] else None,
         "k_weight": _randn(g, D).mul_(0.1).add_(1) if c["norm"] else None,
         "k_cache": _randn(g, pages, c["kv"], page, D, dtype=torch.bfloat16),
         "v_cache": _randn(g, pages, c["kv"], page, D, dtype=torch.bfloat16),
         "q_out": torch.zeros(rows, c["heads"], D, dtype=torch.bfloat16, device=DEV)}
    if own:
        import mtp_speculative_decoding_qmv_gb300 as sv

        s["freqs"] = sv.rope_freqs(s["inv_freq"])
    return s


def _prepare_attend(c, g):
    ctx, new = _lengths(c)
    B, page, D = c["requests"], c["page"], c["dim"]
    total = [n + t for n, t in zip(ctx, new)]
    if c["empty"]:  # a request that was refused its pages keeps its rows, with nothing to attend
        total[1] = 0
    held = [_pages_of(n, page) for n in total]
    most = max(held) + 2
    pages = sum(held) + 1
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    h = _ints(held)
    at = torch.arange(most, device=DEV)[None, :]
    idx = (torch.cumsum(h, 0) - h)[:, None] + at
    table = torch.where(at < h[:, None], ids[idx.clamp(max=pages - 1)], -1).contiguous()
    rows = sum(new)
    start = [0]
    for t in new:
        start.append(start[-1] + t)
    s = {"case": c, "q": _randn(g, rows, c["heads"], D, dtype=torch.bfloat16, std=1.5),
         "k_cache": _randn(g, pages, c["kv"], page, D, dtype=torch.bfloat16),
         "v_cache": _randn(g, pages, c["kv"], page, D, dtype=torch.bfloat16),
         "table": table, "q_start": _ints(start), "kv_len": _ints(total), "max_new": max(new),
         "max_kv": max(1, max(total)), "scale": 1.0 / math.sqrt(D),
         "out": torch.zeros(rows, c["heads"], D, dtype=torch.bfloat16, device=DEV),
         "lse": torch.zeros(rows, c["heads"], device=DEV)}
    if own:
        import mtp_speculative_decoding_qmv_gb300 as sv

        s["workspace"] = sv.make_attention_workspace(D, torch.device(DEV, 0))
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    if own:
        return {"pages": _own_pages, "append": _own_append, "attend": _own_attend}[s["case"]["op"]](s)
    return {"pages": _plain_pages, "append": _plain_append, "attend": _plain_attend}[s["case"]["op"]](s)


def _own_pages(s):
    import mtp_speculative_decoding_qmv_gb300 as sv

    r = sv.kv_pages_step(s["length"], s["held"], s["cursor"], s["ring"], s["table"], s["n_new"],
                         s["page"], s["rows"], n_commit=s["commit"], n_commit_bias=1,
                         length_out=s["length_out"], held_out=s["held_out"],
                         cursor_out=s["cursor_out"], q_start=s["q_start"], kv_len=s["kv_len"],
                         slots=s["slots"], positions=s["positions"], err_flags=s["flags"])
    return (*r, s["table"], s["ring"])


def _own_append(s):
    import mtp_speculative_decoding_qmv_gb300 as sv

    sv.rope_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"],
                      s["k_cache"], s["v_cache"], axis=s["axis"], q_weight=s["q_weight"],
                      k_weight=s["k_weight"], interleaved=s["case"]["pairs"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_attend(s):
    import mtp_speculative_decoding_qmv_gb300 as sv

    sv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"],
                       s["max_new"], scale=s["scale"], window=s["case"]["window"], out=s["out"],
                       lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _plain_pages(s):
    page, rows, table, ring = s["page"], s["rows"], s["table"], s["ring"]
    B, most = table.shape
    P = ring.numel()
    head, n_free = s["cursor"][0].long(), s["cursor"][1].long()
    ended = s["n_new"] < 0
    n = s["n_new"].clamp(min=0).long()
    held = s["held"].long()
    grown = s["length"].long() + s["commit"] + 1
    L = torch.minimum(grown.clamp(min=0), held * page)
    flags = torch.where((L != grown) & ~ended, 16, 0)
    L = torch.where(ended, 0, L)
    ends = torch.cumsum(n, 0)
    q0 = ends - n
    unfit = ends > rows
    want = (L + n + page - 1) // page
    long = want > most
    need = torch.where(unfit | long | ended, 0, (want - held).clamp(min=0))
    taken = torch.cumsum(need, 0)
    short = (need > 0) & (taken > n_free)
    refused = unfit | long | short
    flags = flags | torch.where(long | short, 32, 0) | torch.where(unfit, 64, 0)
    got = torch.where(short, 0, need)
    first = taken - need
    at = torch.arange(most, device=table.device)[None, :]
    fresh = (at >= held[:, None]) & (at < (held + got)[:, None])
    from_ring = ring[(head + first[:, None] + (at - held[:, None])) % P]
    table.copy_(torch.where(fresh, from_ring, table))
    back = torch.where(ended, held, 0)
    freed = torch.cumsum(back, 0)
    # entry i of the freed pages: request `who`, its page `which`; the ring keeps its others
    i = torch.arange(P, device=table.device)
    who = torch.searchsorted(freed, i, right=True).clamp(max=B - 1)
    which = (i - (freed - back)[who]).clamp(0, most - 1)
    to = (head + n_free + i) % P
    ring[to] = torch.where(i < freed[-1], table[who, which], ring[to])
    used = got.sum()
    cursor = torch.stack([(head + used) % P, (n_free - used + freed[-1]).clamp(max=P)]).int()
    r = torch.arange(rows, device=table.device)
    b = torch.searchsorted(ends, r, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = L[b] + r - q0[b]
    pg = table[b, (pos // page).clamp(max=most - 1)].long()
    ok = real & ~refused[b] & (pg >= 0) & (pg < P)
    slots = torch.where(ok, pg * page + pos % page, -1).int()
    positions = torch.where(real, pos, 0).int()
    q_start = torch.cat([ends.new_zeros(1), ends]).clamp(max=rows).int()
    kv_len = torch.where(refused, 0, L + n).int()
    held_out = torch.where(ended, 0, held + got).int()
    return L.int(), held_out, cursor, q_start, kv_len, slots, positions, flags.int(), table, ring


def _plain_rotate(c, x, weight, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight
    half = c["rot"] // 2
    if c["pairs"]:
        a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:c["rot"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., c["rot"]:]], -1).bfloat16()


def _plain_append(s):
    c = s["case"]
    pos = s["positions"].double()
    angle = (pos[:, s["axis"].long()] if s["axis"] is not None else pos[:, :1]) * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    s["q_out"].copy_(_plain_rotate(c, s["q"], s["q_weight"], cos, sin))
    k = _plain_rotate(c, s["k"], s["k_weight"], cos, sin)
    v = s["v"].bfloat16()
    # a padding row writes what the first real row writes, to the same place
    real = s["slots"] >= 0
    i = torch.where(real, torch.arange(c["rows"], device=DEV), real.int().argmax())
    slot = s["slots"][i].long()
    s["k_cache"][slot // c["page"], :, slot % c["page"]] = k[i]
    s["v_cache"][slot // c["page"], :, slot % c["page"]] = v[i]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    c = s["case"]
    B, Hkv, D, N, T = c["requests"], c["kv"], c["dim"], s["max_new"], s["max_kv"]
    G = c["heads"] // Hkv
    start, L = s["q_start"].long(), s["kv_len"].long()
    n = start[1:] - start[:-1]
    t, j = torch.arange(N, device=DEV), torch.arange(T, device=DEV)
    rows = (start[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D)
    pages = s["table"][:, :_pages_of(T, c["page"])].clamp(min=0).long()

    def gather(cache):
        x = cache[pages].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :T].float()
        return torch.where((j < L[:, None])[:, None, :, None], x, 0.0)

    limit = (L - n)[:, None] + t  # the last position that each row may attend
    allowed = (j <= limit[..., None]) & (j < L[:, None, None])
    if c["window"]:
        allowed &= j > limit[..., None] - c["window"]
    x = (q @ gather(s["k_cache"]).transpose(2, 3)).view(B, Hkv, G, N, T).mul_(s["scale"])
    x = torch.where(allowed[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * N, T) @ gather(s["v_cache"])).view(B, Hkv, G, N, D)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (m + total.log()).squeeze(-1)  # -inf where nothing is attended
    r = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(start[1:], r, right=True)
    at = r - start[b]
    o = o.permute(0, 3, 1, 2, 4)[b, at].reshape(-1, c["heads"], D)
    lse = lse.permute(0, 3, 1, 2)[b, at].reshape(-1, c["heads"])
    s["out"].copy_(o)
    s["lse"].copy_(lse)
    return s["out"], s["lse"]


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "pages":
        ctx, _, new = _step_lengths(c)
        held = [_pages_of(n, c["page"]) for n in ctx]
        moved = sum(max(0, _pages_of(n + t, c["page"]) - h) if t > 0 else h if t < 0 else 0
                    for n, t, h in zip(ctx, new, held))
        rows = sum(t for t in new if t > 0) + 5
        # four words read and five written for a request, a page id moved, a row's slot and position
        return {"bytes": 4.0 * (9 * c["requests"] + 2 * moved + 2 * rows), "flops": 0.0}
    if c["op"] == "append":
        size = 4 if c["dtype"] == "f32" else 2
        values = c["rows"] * (c["heads"] + 2 * c["kv"]) * c["dim"]
        turned = c["rows"] * (c["heads"] + c["kv"])
        return {"bytes": values * (size + 2.0) + c["rows"] * 4.0 * (c["axes"] + 1),
                "flops": turned * (3.0 * c["rot"] + (4.0 * c["dim"] if c["norm"] else 0.0))}
    ctx, new = _lengths(c)
    pairs = read = 0
    for b, (n, t) in enumerate(zip(ctx, new)):
        if c["empty"] and b == 1:
            continue
        w = c["window"] or n + t
        pairs += sum(min(n + i + 1, w) for i in range(t))
        read += min(n + t, w + t - 1)
    rows = sum(new)
    return {"bytes": 4.0 * read * c["kv"] * c["dim"] + rows * c["heads"] * (4.0 * c["dim"] + 4.0),
            "flops": 4.0 * pairs * c["heads"] * c["dim"]}


# ----------------------------------------------------------------------------
# the definitions, in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers: the plain form's are held to exactly
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)


def _exact_append(c, s):
    D, R, half, page = c["dim"], c["rot"], c["rot"] // 2, c["page"]
    freq, pos = s["inv_freq"], s["positions"].double()
    # every element e of a head as a sum of two of its inputs: itself and its partner
    e = torch.arange(R, device=DEV)
    pair = e // 2 if c["pairs"] else e % half
    partner = (e ^ 1) if c["pairs"] else (e + half) % R
    sign = torch.where((e % 2 == 0) if c["pairs"] else (e < half), -1.0, 1.0).double()
    turns = torch.empty(c["rows"], R, dtype=torch.float64, device=DEV)
    for i in range(R):
        f = int(pair[i])
        turns[:, i] = pos[:, int(s["axis"][f]) if s["axis"] is not None else 0] * freq[f]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        z = y.clone()
        z[..., :R] = y[..., :R] * turns.cos()[:, None] + y[..., partner] * sign * turns.sin()[:, None]
        out.append(z)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    v = s["v"].double()
    keep = torch.tensor([r for r, slot in enumerate(s["slots"].tolist()) if slot >= 0], device=DEV)
    slot = s["slots"].long()[keep]
    k_cache[slot.div(page, rounding_mode="floor"), :, slot % page] = out[1][keep]
    v_cache[slot.div(page, rounding_mode="floor"), :, slot % page] = v[keep]
    return out[0], k_cache, v_cache


def _exact_attend(c, s):
    ctx, new = _lengths(c)
    D, G = c["dim"], c["heads"] // c["kv"]
    if work(c)["flops"] > 4e12:
        return None
    out = torch.zeros(sum(new), c["heads"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((sum(new), c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    row = 0
    for b in range(c["requests"]):
        first, row = row, row + new[b]
        total = int(s["kv_len"][b])
        if total == 0:
            continue
        held = s["table"][b, :_pages_of(total, c["page"])].long()
        for h in range(c["kv"]):
            k = s["k_cache"][held, h].reshape(-1, D)[:total].double()
            v = s["v_cache"][held, h].reshape(-1, D)[:total].double()
            for t0 in range(0, new[b], 512):
                t1 = min(new[b], t0 + 512)
                last = ctx[b] + t1  # no row of this piece attends further
                low = max(0, ctx[b] + t0 - c["window"] + 1) if c["window"] else 0
                at = torch.arange(low, last, device=DEV)
                mine = ctx[b] + torch.arange(t0, t1, device=DEV)[:, None, None]
                hidden = at > mine
                if c["window"]:
                    hidden = hidden | (mine - at >= c["window"])
                q = s["q"][first + t0:first + t1, h * G:(h + 1) * G].double()
                z = torch.einsum("tgd,jd->tgj", q, k[low:last]) * s["scale"]
                z.masked_fill_(hidden, -math.inf)
                lse[first + t0:first + t1, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[first + t0:first + t1, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[low:last]
    return out, lse
