"""One attention layer of a target model through a few speculative cycles.

Prompts of different lengths go in as one packed chunk; then every cycle
verifies K drafts a request: the 4-bit projections (qmv_wide, qmv_smallm), the
step's pages and slots (kv_pages_step), rotary positions and cache writes
(rope_kv_append), attention over the pages (paged_attention) and acceptance
(spec_accept), whose accepted counts commit the next cycle's lengths on the
device.  The cycle is one CUDA graph, replayed; nothing waits for the host.
Weights, embeddings and logits are random.

    python examples/attention_layer.py [--cycles 6] [--check]

--check recomputes the last cycle's attention from the committed tokens' own
projections, densely in float64.
"""
from __future__ import annotations

import argparse
import math
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))

import mtp_speculative_decoding_qmv_gb300 as sv  # noqa: E402

HIDDEN, HQ, HKV, D, PAGE, K, VOCAB = 1024, 8, 2, 128, 16, 3, 4096


def quantised(n_out: int, n_in: int, g: torch.Generator):
    w = torch.randn(n_out, n_in, generator=g, device=g.device) / math.sqrt(n_in)
    return sv.qmv_requantize(w.bfloat16())


class AttentionLayer:
    """Weights, the paged cache and its bookkeeping, for up to ``requests``."""

    def __init__(self, requests: int, pages: int, most_pages: int, g: torch.Generator):
        dev = g.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.qkv = quantised((HQ + 2 * HKV) * D, HIDDEN, g)
        self.o = quantised(HIDDEN, HQ * D, g)
        self.q_weight = torch.ones(D, device=dev)
        self.k_weight = torch.ones(D, device=dev)
        exps = torch.arange(D // 2, dtype=torch.float64, device=dev)
        self.freqs = sv.rope_freqs(1e6 ** (-2.0 * exps / D))
        self.k_cache = torch.zeros(pages, HKV, PAGE, D, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.length = torch.zeros(requests, **i32)
        self.held = torch.zeros(requests, **i32)
        self.ring = torch.arange(pages, **i32)
        self.cursor = torch.tensor([0, pages], **i32)
        self.table = torch.zeros(requests, most_pages, **i32)
        self.workspace = sv.make_attention_workspace(D, dev)

    def project(self, weights, x: torch.Tensor) -> torch.Tensor:
        if x.shape[0] <= 16:
            return sv.qmv_smallm(*weights, x)
        return torch.cat([sv.qmv_wide(*weights, part) for part in x.split(128)])

    def step(self, x: torch.Tensor, n_new: torch.Tensor, max_new: int,
             n_commit: torch.Tensor | None, bias: int):
        """x bf16 [rows, HIDDEN], the packed rows of n_new tokens a request,
        after n_commit + bias tokens of the step before are committed.  Returns
        the layer's output, the attention's and the step's bookkeeping."""
        s = sv.kv_pages_step(self.length, self.held, self.cursor, self.ring, self.table, n_new,
                             PAGE, x.shape[0], n_commit=n_commit, n_commit_bias=bias,
                             length_out=self.length, held_out=self.held, cursor_out=self.cursor)
        rows = self.project(self.qkv, x).view(-1, HQ + 2 * HKV, D)
        q = sv.rope_kv_append(rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:], s.positions,
                              s.slots, self.freqs, self.k_cache, self.v_cache,
                              q_weight=self.q_weight, k_weight=self.k_weight)
        attended, _ = sv.paged_attention(q, self.k_cache, self.v_cache, self.table, s.q_start,
                                         s.kv_len, max_new, workspace=self.workspace)
        return self.project(self.o, attended.view(-1, HQ * D)), attended, s


def dense(layer: AttentionLayer, history: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
    """Attention of one request's rows x after the tokens of ``history``
    (embeddings), from the projections, in float64."""
    tokens = torch.cat([history, x])
    rows = layer.project(layer.qkv, tokens).double().view(-1, HQ + 2 * HKV, D)
    pos = torch.arange(len(tokens), device=x.device, dtype=torch.float64)
    exps = torch.arange(D // 2, dtype=torch.float64, device=x.device)
    angle = pos[:, None, None] * 1e6 ** (-2.0 * exps / D)

    def turn(h):
        h = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        a, b = h[..., :D // 2], h[..., D // 2:]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    q, k, v = turn(rows[:, :HQ]), turn(rows[:, HQ:HQ + HKV]), rows[:, HQ + HKV:]
    k, v = (t.repeat_interleave(HQ // HKV, 1) for t in (k, v))
    scores = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
    scores = scores.masked_fill(pos[None, None, :] > pos[None, :, None], -math.inf)
    return torch.einsum("hij,jhd->ihd", scores.softmax(-1), v)[len(history):]


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cycles", type=int, default=6)
    ap.add_argument("--check", action="store_true")
    args = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    prompts = [37, 5, 120, 64]
    B, rows = len(prompts), len(prompts) * (K + 1)
    layer = AttentionLayer(B, pages=64, most_pages=32, g=g)

    def embed(n):
        return torch.randn(n, HIDDEN, generator=g, device=dev).bfloat16()

    # the prompts, one packed chunk; they are committed by the first cycle
    chunk = embed(sum(prompts))
    n_new = torch.tensor(prompts, dtype=torch.int32, device=dev)
    layer.step(chunk, n_new, max(prompts), None, 0)
    layer.length.copy_(n_new)
    history = [list(part) for part in chunk.split(prompts)]

    # a cycle's fixed buffers; the first one commits nothing (-1 + 1)
    x = torch.empty(rows, HIDDEN, dtype=torch.bfloat16, device=dev)
    n_new = torch.full((B,), K + 1, dtype=torch.int32, device=dev)
    target = torch.empty(B, K + 1, VOCAB, device=dev)
    draft = torch.empty(B, K, VOCAB, device=dev)
    drafts = torch.empty(B, K, dtype=torch.int32, device=dev)
    u_accept, u_sample = torch.empty(B, K, device=dev), torch.empty(B, device=dev)
    accepted = torch.full((B,), -1, dtype=torch.int32, device=dev)
    accept_ws = sv.make_accept_workspace(B, K, VOCAB, dev)

    def cycle():
        out = layer.step(x, n_new, K + 1, accepted, 1)
        sv.spec_accept(target, draft, drafts, u_accept, u_sample, 0.6, 20, 0.95,
                       workspace=accept_ws, n_accepted=accepted)
        return out

    def inputs():
        x.copy_(embed(rows))
        draft.normal_(generator=g).mul_(3.0)
        target[:, :K].copy_(draft)
        target[:, K].normal_(generator=g)
        target.add_(torch.randn(target.shape, generator=g, device=dev), alpha=0.7)
        drafts.copy_(draft.argmax(-1))
        u_accept.uniform_(generator=g)
        u_sample.uniform_(generator=g)

    inputs()
    state = [t.clone() for t in (layer.length, layer.held, layer.cursor, layer.ring, layer.table)]
    side = torch.cuda.Stream()  # a first run outside the graph
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cycle()
    torch.cuda.current_stream().wait_stream(side)
    for t, saved in zip((layer.length, layer.held, layer.cursor, layer.ring, layer.table), state):
        t.copy_(saved)
    accepted.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, attended, step = cycle()

    worst = 0.0
    for i in range(args.cycles):
        if i:
            inputs()
        graph.replay()
        if args.check and i == args.cycles - 1:
            for b in range(B):
                want = dense(layer, torch.stack(history[b]), x[b * (K + 1):(b + 1) * (K + 1)])
                got = attended[b * (K + 1):(b + 1) * (K + 1)].double()
                worst = max(worst, float((got - want).norm() / want.norm()))
        taken = accepted.tolist()  # only to follow the tokens here
        for b in range(B):
            history[b] += list(x[b * (K + 1):b * (K + 1) + taken[b] + 1].clone())
        print(f"cycle {i}: lengths {step.length.tolist()}, accepted {taken}, "
              f"flags {step.err_flags.tolist()}")
        assert step.length.tolist() == [len(h) - t - 1 for h, t in zip(history, taken)]
    sv.device_status()
    if args.check:
        print(f"last cycle's attention against float64: relative error {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
