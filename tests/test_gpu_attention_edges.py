"""paged_attention where a CTA goes from one item to the next: split requests
beside refused ones."""
import math

import pytest
import torch

import attention_ref as ref
from gpu_util import dev, sv_module
from test_gpu_paged_attention import _dense

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


class Long:
    """Requests of (context, new tokens) drawn on the device, each with pages of
    its own; a context of None is a refused request: its rows stay, kv_len is 0."""

    def __init__(self, D, Hq, Hkv, page, requests, seed):
        d = dev()
        g = torch.Generator(device=d)
        g.manual_seed(seed)
        self.requests, self.page = requests, page
        held = [0 if ctx is None else -(-(ctx + n) // page) for ctx, n in requests]
        self.k, self.v = (torch.randn(sum(held), Hkv, page, D, generator=g, device=d,
                                      dtype=torch.bfloat16) for _ in range(2))
        self.table = torch.zeros(len(held), max(held), dtype=torch.int32, device=d)
        ids = torch.randperm(sum(held), generator=g, device=d).to(torch.int32)
        for b, n in enumerate(held):
            self.table[b, :n], ids = ids[:n], ids[n:]
        starts = [0]
        for _, n in requests:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.q = torch.randn(starts[-1], Hq, D, generator=g, device=d, dtype=torch.bfloat16) * 1.5
        self.q_start = torch.tensor(starts, dtype=torch.int32, device=d)
        self.kv_len = torch.tensor([0 if ctx is None else ctx + n for ctx, n in requests],
                                   dtype=torch.int32, device=d)
        self.scale = 1.0 / math.sqrt(D)

    def args(self):
        return self.q, self.k, self.v, self.table, self.q_start, self.kv_len

    def want(self, b):
        """Request b's rows in float64: out, lse."""
        ctx, n = self.requests[b]
        return _dense(self.q[self.starts[b]:self.starts[b + 1]], self.k, self.v,
                      self.table[b:b + 1], self.page, ctx, n, self.scale)


def _close(got, want):
    # weights and outputs are rounded to bf16 (2^-8 at most each, in norm as well)
    return float((got.double() - want).norm() / want.norm()) < 2 * ref.HALF_BF16


@pytest.mark.parametrize("D,Hq,new,ctx", [(64, 1, 20, 400000), (128, 1, 30, 400000),
                                          (128, 1, 129, 100000), (64, 4, 200, 30000),
                                          (256, 1, 20, 400000), (256, 1, 70, 60000)])
def test_a_refused_request_after_a_split_one(sv, D, Hq, new, ctx):
    """The CTA that joins a split item goes on to rows without keys, whose zeros
    go through the shared memory that the join's weights lie in."""
    c = Long(D, Hq, 1, 64, [(ctx, new), (None, 300), (ctx // 2, new), (None, 40), (900, 3)], D + new)
    ws = sv.make_attention_workspace(D, dev())
    lse = torch.empty(c.q.shape[:2], device=dev())
    out = sv.paged_attention(*c.args(), 300, lse=lse, workspace=ws)[0].clone()
    for b, (context, _) in enumerate(c.requests):
        rows = slice(c.starts[b], c.starts[b + 1])
        if context is None:
            assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
        else:
            assert _close(out[rows], c.want(b)[0]), b
    for _ in range(100):
        assert torch.equal(sv.paged_attention(*c.args(), 300, workspace=ws)[0], out)
    sv.device_status()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_items_with_infinities_one_after_another(sv, D):
    """Many short requests whose newest value is infinite, several a CTA: each
    item finds its own."""
    d = dev()
    B, new, Hq = 700, 5, 15  # 75 rows of one kv head
    c = Long(D, Hq, 1, 16, [(11, new)] * B, D)
    clean = c.v.clone()
    page, offset = c.table[:, 0].long(), 15
    odd = torch.arange(B, device=d) % 3 != 1
    c.v[page[odd], 0, offset, ::7] = math.inf
    ws = sv.make_attention_workspace(D, d)
    scale = c.scale
    k, v = (t[page, 0].double() for t in (c.k, clean))  # [B, 16, D]
    q = c.q.view(B, new, Hq, D).double()
    x = torch.einsum("btgd,bjd->btgj", q, k) * scale
    at = torch.arange(16, device=d)
    x = x.masked_fill(at > 11 + torch.arange(new, device=d)[:, None, None], -math.inf)
    want = torch.einsum("btgj,bjd->btgd", x.softmax(-1), v)
    infinite = torch.zeros_like(want, dtype=torch.bool)
    infinite[odd, new - 1, :, ::7] = True  # seen by the last row alone
    for _ in range(20):
        out = sv.paged_attention(*c.args(), 100, workspace=ws)[0].view(B, new, Hq, D).double()
        assert torch.equal(torch.isposinf(out), infinite)
        assert _close(out[~infinite], want[~infinite])
