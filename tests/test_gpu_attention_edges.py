"""paged_attention where a CTA goes from one item to the next: split requests
beside refused ones, non-finite values that some rows attend and others do not."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref
from gpu_util import dev, sv_module
from test_gpu_paged_attention import Case, _dense

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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [4, 30, 100, 150])  # with G = 2: row tiles of 16 to 256, two items
@pytest.mark.parametrize("window", [0, 20, 130])
def test_non_finite_values_reach_the_rows_that_attend_them(sv, D, new, window):
    """Infinities of both signs and NaN in the first and last places of the rows:
    the same places are infinite and NaN as in float64, the others as exact as
    ever."""
    c = Case(D, 4, 2, 32, [340, 5], [new, 2], seed=D + new + window)
    first = 340 - new
    places = [339, 338, first + 1, first + new // 2]
    if window:
        places += [max(0, first - window + 3), max(0, first + new // 2 - window + 1)]
    for i, j in enumerate(places):
        p, o = c.table[0, j // 32], j % 32
        c.v[p, :, o, i::7] = [math.inf, -math.inf, math.nan][i % 3]
        c.v[p, 1, o, 5] = math.inf  # of several positions
        c.v[p, 1, o, 6] = math.inf if i % 2 else -math.inf
    c.k[c.table[0, 338 // 32], 0, 338 % 32] = -math.inf  # weight zero, or NaN
    t = c.device()
    lse = torch.empty(c.rows, 4, device=dev())
    out, _ = sv.paged_attention(*t, new, scale=c.scale, window=window, lse=lse)
    sv.device_status()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, want_lse, mag, smag = c.want(window)
    assert np.array_equal(np.isnan(out), np.isnan(want))
    infinite = np.isinf(want)
    assert infinite.any() and np.array_equal(infinite, np.isinf(out))
    assert np.array_equal(out[infinite], want[infinite])
    keep = np.isfinite(smag).all(1)  # rows whose scores are finite
    assert keep.sum() > 2
    zero = lambda a: np.where(infinite, 0.0, a)[keep]  # noqa: E731
    ref.check_attention(zero(out), lse[keep],
                        (zero(want), want_lse[keep], zero(mag), smag[keep]), D, 340)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [60, 100])
def test_an_infinity_in_a_long_context(sv, D, new):
    """The newest token's value is infinite in every head of a context of 250,000:
    the rows that do not attend it and the items after it are as without it."""
    H, ctx = 40, 250000
    c = Long(D, H, H, 128, [(ctx, new)], D)
    clean = c.v.clone()
    page, offset = int(c.table[0, (ctx + new - 1) // 128]), (ctx + new - 1) % 128
    c.v[page, :, offset, ::3] = math.inf
    out = sv.paged_attention(*c.args(), new)[0]
    sv.device_status()
    infinite = torch.zeros(new, 1, D, dtype=torch.bool, device=dev())
    infinite[-1, :, ::3] = True
    assert torch.equal(torch.isposinf(out), infinite.expand(new, H, D))
    for h in (0, 1, 17, 38, 39):
        want, _ = _dense(c.q[:, h:h + 1], c.k[:, h:h + 1], clean[:, h:h + 1], c.table, 128, ctx,
                         new, c.scale)
        assert _close(out[:, h:h + 1][~infinite], want[~infinite]), h


def _none(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=dev())


def test_a_step_without_requests(sv):
    """Its rows have no slots, and the cursor is carried on."""
    cursor = torch.tensor([3, 5], dtype=torch.int32, device=dev())
    given = {k: _none(n) + 9 for k, n in
             (("cursor_out", 2), ("q_start", 1), ("slots", 6), ("positions", 6))}
    step = sv.kv_pages_step(_none(0), _none(0), cursor, _none(8), _none(0, 4), _none(0), 16, 6,
                            **given)
    assert step.cursor.tolist() == [3, 5] and step.q_start.tolist() == [0]
    assert step.slots.tolist() == [-1] * 6 and step.positions.tolist() == [0] * 6
    step = sv.kv_pages_step(_none(0), _none(0), cursor, _none(8), _none(0, 4), _none(0), 16, 6,
                            cursor_out=cursor)
    assert step.cursor is cursor and cursor.tolist() == [3, 5]


@pytest.mark.parametrize("D", [64, 256])
def test_rows_without_requests_attend_nothing(sv, D):
    q = torch.ones(6, 4, D, dtype=torch.bfloat16, device=dev())
    cache = torch.ones(8, 2, 16, D, dtype=torch.bfloat16, device=dev())
    out, lse = torch.full_like(q, 7.0), torch.full((6, 4), 7.0, device=dev())
    for rows in (6, 0):
        got, got_lse = sv.paged_attention(q[:rows], cache, cache, _none(0, 4), _none(1), _none(0),
                                          4, out=out[:rows], lse=lse[:rows])
        assert (got == 0).all() and torch.isneginf(got_lse).all() and len(got) == rows


def test_two_streams_at_once(sv):
    """Calls of both families side by side, each stream with its workspace: the
    bits of calls one after another."""
    d = dev()
    cases = [(Long(128, 8, 2, 16, [(9000, 300), (None, 5), (200, 40)], 1), 300),
             (Long(128, 8, 2, 64, [(20000, 4), (300, 1), (7, 4)], 2), 4)]
    work = []
    for c, most in cases:
        ws = sv.make_attention_workspace(128, d)
        out = torch.empty_like(c.q)
        sv.paged_attention(*c.args(), most, out=out, workspace=ws)
        work.append((c, most, ws, out.clone(), [torch.empty_like(out) for _ in range(30)],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(30):
        for c, most, ws, _, outs, stream in work:
            with torch.cuda.stream(stream):
                sv.paged_attention(*c.args(), most, out=outs[i], workspace=ws)
    torch.cuda.synchronize()
    sv.device_status()
    for _, _, _, want, outs, _ in work:
        assert all(torch.equal(o, want) for o in outs)


def test_the_calls_allocate_nothing(sv):
    d = dev()
    B, rows, page, D = 3, 7, 16, 64
    i32 = dict(dtype=torch.int32, device=d)
    length, held, cursor = _none(B), _none(B), torch.tensor([0, 64], **i32)
    ring, table, n_new = torch.arange(64, **i32), _none(B, 8), torch.tensor([4, 1, 2], **i32)
    commit = torch.tensor([1, 1, 1], **i32)
    kw = dict(length_out=length, held_out=held, cursor_out=cursor, q_start=_none(B + 1),
              kv_len=_none(B), slots=_none(rows), positions=_none(rows), err_flags=_none(B))
    x = torch.randn(rows, 8, D, device=d)
    cache = torch.zeros(2, 64, 2, page, D, dtype=torch.bfloat16, device=d)
    freqs = sv.rope_freqs(torch.ones(8, dtype=torch.float64, device=d))
    q, out = (torch.empty(rows, 4, D, dtype=torch.bfloat16, device=d) for _ in range(2))
    lse, ws = torch.empty(rows, 4, device=d), sv.make_attention_workspace(D, d)

    def step():
        s = sv.kv_pages_step(length, held, cursor, ring, table, n_new, page, rows, n_commit=commit,
                             **kw)
        sv.rope_kv_append(x[:, :4], x[:, 4:6], x[:, 6:], s.positions, s.slots, freqs, cache[0],
                          cache[1], q_out=q)
        for most in (4, 100):  # both families
            sv.paged_attention(q, cache[0], cache[1], table, s.q_start, s.kv_len, most, out=out,
                               lse=lse, workspace=ws)

    def held_memory():
        torch.cuda.synchronize()
        return (torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0])

    step()
    before = held_memory()
    for _ in range(5):
        step()
    assert held_memory() == before
    assert torch.isfinite(out.float()).all()
