"""paged_attention against float64, row by row (bounds in attention_ref)."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref
from gpu_util import dev, sv_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


class Case:
    """Caches whose unused slots and pages are all NaN, block tables whose
    entries past a request's pages are out of range."""

    def __init__(self, D, Hq, Hkv, page, lens, news, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.news, self.page = lens, news, page
        B = len(lens)
        held = [-(-n // page) for n in lens]
        pages = sum(held) + 3
        ids = rng.permutation(pages)
        self.table = np.full((B, max(held + [1]) + 1), 1 << 30, np.int32)
        self.table[:, -1] = -1
        self.k = np.full((pages, Hkv, page, D), np.nan, np.float32)
        self.v = np.full((pages, Hkv, page, D), np.nan, np.float32)
        at = 0
        for b in range(B):
            self.table[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
            for j in range(lens[b]):
                p = self.table[b, j // page]
                self.k[p, :, j % page] = rng.normal(size=(Hkv, D))
                self.v[p, :, j % page] = rng.normal(size=(Hkv, D))
        self.q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.rows = int(self.q_start[-1])
        self.q = (rng.normal(size=(self.rows, Hq, D)) * spread).astype(np.float32)
        for n in ("q", "k", "v"):  # the values that bf16 holds
            setattr(self, n, torch.from_numpy(getattr(self, n)).bfloat16().float().numpy())
        self.scale = 1.0 / math.sqrt(D)

    def device(self):
        d = dev()
        bf = lambda a: torch.from_numpy(a).bfloat16().to(d)  # noqa: E731
        return (bf(self.q), bf(self.k), bf(self.v), torch.from_numpy(self.table).to(d),
                torch.from_numpy(self.q_start).to(d),
                torch.tensor(self.lens, dtype=torch.int32, device=d))

    def want(self, window=0):
        return ref.attention(self.q, self.k, self.v, self.table, self.q_start, self.lens,
                             float(np.float32(self.scale)), window)

    def check(self, sv, window=0, max_new=None):
        t = self.device()
        lse = torch.full((self.rows, self.q.shape[1]), 5.0, device=dev())
        ws = sv.make_attention_workspace(self.q.shape[2], dev())
        out, _ = sv.paged_attention(*t, max(self.news) if max_new is None else max_new,
                                    scale=self.scale, window=window, lse=lse, workspace=ws)
        assert int(torch.count_nonzero(ws[:4096])) == 0
        sv.device_status()
        ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                            self.want(window), self.q.shape[2], max(self.lens))
        return out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens_and_verify_blocks(sv, D, page):
    Case(D, 10, 2, page, [1, 5, 63, 64, 65, 200, 0, 130], [1, 4, 4, 1, 4, 3, 0, 4], seed=D).check(sv)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 16, 1), (128, 3, 1), (256, 40, 2),
                                      (64, 70, 1), (128, 1, 1)])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_head_layouts(sv, D, Hq, Hkv, page):
    Case(D, Hq, Hkv, page, [37, 300, 90], [2, 5, 1], seed=Hq).check(sv)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,news", [
    ([300], [300]), ([517, 64, 1, 129], [130, 64, 1, 128]), ([700, 33], [257, 1]),
    ([40, 500, 260], [39, 3, 260]), ([1025], [513]), ([128, 128, 256], [128, 1, 129])])
def test_chunks_of_prompts(sv, D, lens, news):
    Case(D, 4, 2, 32, lens, news, seed=sum(lens) + D).check(sv)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("window", [1, 17, 64, 200, 5000])
def test_windows(sv, D, window, page):
    Case(D, 6, 2, page, [400, 70, 9, 513], [4, 1, 9, 2], seed=window).check(sv, window)
    Case(D, 5, 1, page, [400, 333], [150, 90], seed=window + 1).check(sv, window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_attend_nothing(sv, D):
    c = Case(D, 4, 2, 16, [0, 3, 50, 0], [2, 7, 3, 90])
    out = c.check(sv)
    assert (out[:2] == 0).all() and (out[2:6] == 0).all() and (out[12:] == 0).all()
    assert (out[6] != 0).any()


def test_max_new_is_only_a_bound(sv):
    for D in (64, 128):
        c = Case(D, 4, 2, 16, [150, 40], [90, 3])
        for bound in (1, 8, 90, 4000):
            c.check(sv, max_new=bound)


def test_rows_past_the_last_are_zero(sv):
    d = dev()
    for news in ([2, 3], [70, 3]):
        c = Case(128, 4, 2, 16, [100, 40], news)
        q, k, v, table, qs, kl = c.device()
        q = torch.cat([q, torch.ones(5, 4, 128, device=d, dtype=torch.bfloat16)])
        lse = torch.zeros(c.rows + 5, 4, device=d)
        out = torch.ones_like(q)
        sv.paged_attention(q, k, v, table, qs, kl, max(news), out=out, lse=lse)
        assert (out[c.rows:] == 0).all() and torch.isneginf(lse[c.rows:]).all()
        assert torch.isfinite(lse[:c.rows]).all()


@pytest.mark.parametrize("D,news", [(64, [4]), (128, [1]), (256, [4]), (128, [40]), (64, [70]),
                                    (128, [130]), (256, [130])])
def test_one_long_request_is_split_and_joined(sv, D, news):
    Case(D, 5, 1, 64, [9001], news, seed=D, spread=2.0).check(sv)


@pytest.mark.parametrize("D,news", [(128, 4), (64, 70), (128, 70)])
def test_deterministic(sv, D, news):
    c = Case(D, 8, 2, 16, [3000, 2, 777], [news, 1, news], seed=4)
    t = c.device()
    ws = sv.make_attention_workspace(D, dev())
    first = sv.paged_attention(*t, news, workspace=ws)[0].clone()
    for _ in range(20):
        assert torch.equal(sv.paged_attention(*t, news, workspace=ws)[0], first)


@pytest.mark.parametrize("D,new", [(64, 4), (128, 4), (256, 4), (64, 100), (128, 100), (256, 100)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_masked_non_finite_values_have_no_effect(sv, D, new, what):
    """The last token of the chunk holds non-finite keys and values: only the
    last row may see them.  Before the window, likewise."""
    c = Case(D, 4, 2, 32, [260, 90], [new, 1], seed=3)
    clean = c.want()
    p, o = c.table[0, 259 // 32], 259 % 32
    c.v[p, :, o, ::3] = what
    c.k[p, 0, o, 1] = what
    t = c.device()
    lse = torch.empty(c.rows, 4, device=dev())
    out, _ = sv.paged_attention(*t, new, scale=c.scale, lse=lse)
    keep = [r for r in range(c.rows) if r != new - 1]
    ref.check_attention(out[keep].double().cpu().numpy(), lse[keep].double().cpu().numpy(),
                        [a[keep] for a in clean], D, 260)
    assert (~torch.isfinite(out[new - 1, :, ::3])).all()
    # before the window of every row but the first
    c = Case(D, 4, 2, 32, [260], [new], seed=5)
    first = 260 - new - 20 + 1
    p, o = c.table[0, first // 32], first % 32
    clean = c.want(20)
    c.v[p, :, o] = what
    t = c.device()
    out, _ = sv.paged_attention(*t, new, scale=c.scale, window=20)
    ref.check_attention(out[1:].double().cpu().numpy(), None, [a[1:] for a in clean], D, 260)
    assert (~torch.isfinite(out[0])).all()


@pytest.mark.parametrize("D,new", [(128, 2), (128, 80), (64, 80), (256, 80)])
def test_pages_out_of_range_read_as_zeros(sv, D, new):
    c = Case(D, 4, 2, 16, [200], [new], seed=6)
    c.table[0, 2], c.table[0, 5], c.table[0, 7] = -1, 1 << 30, c.k.shape[0]
    c.check(sv)


@pytest.mark.parametrize("new", [3, 70])
def test_strided_rows_and_another_stream(sv, new):
    d = dev()
    c = Case(128, 4, 2, 16, [200, 31], [new, 1], seed=7)
    q, k, v, table, qs, kl = c.device()
    wide = torch.full((c.rows, 9, 128), math.nan, device=d, dtype=torch.bfloat16)
    wide[:, 2:6] = q
    outs = torch.full((c.rows, 7, 128), 3.0, device=d, dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = sv.make_attention_workspace(128, d)
        sv.paged_attention(wide[:, 2:6], k, v, table, qs, kl, new, scale=c.scale,
                           out=outs[:, 1:5], workspace=ws)
    s.synchronize()
    ref.check_attention(outs[:, 1:5].double().cpu().numpy(), None, c.want(), 128, 200)
    assert (outs[:, 0] == 3).all() and (outs[:, 5:] == 3).all()


@pytest.mark.parametrize("new", [4, 70])
def test_captured_with_growing_lengths(sv, new):
    d = dev()
    c = Case(128, 4, 2, 16, [900, 500], [new, 1], seed=8)
    q, k, v, table, qs, kl = c.device()
    out = torch.empty_like(q)
    ws = sv.make_attention_workspace(128, d)
    sv.paged_attention(q, k, v, table, qs, kl, new, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.paged_attention(q, k, v, table, qs, kl, new, out=out, workspace=ws)
    for lens in ([900, 500], [120, 33], [899, 1], [71, 500]):
        kl.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        c.lens = lens
        ref.check_attention(out.double().cpu().numpy(), None, c.want(), 128, 900)


@pytest.mark.parametrize("new", [1, 80])
def test_offsets_past_32_bits(sv, new):
    d = dev()
    pages, Hkv, page, D = 70000, 4, 64, 128  # 2.3e9 elements a cache
    kc = torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=d)
    vc = torch.zeros_like(kc)
    c = Case(D, 4, Hkv, page, [150], [new], seed=9)
    far = [pages - 1, 65541, 68000]
    for i, p in enumerate(far):
        kc[p] = torch.from_numpy(c.k[c.table[0, i]]).bfloat16().to(d)
        vc[p] = torch.from_numpy(c.v[c.table[0, i]]).bfloat16().to(d)
    q, _, _, _, qs, kl = c.device()
    table = torch.tensor([far], dtype=torch.int32, device=d)
    out, _ = sv.paged_attention(q, kc, vc, table, qs, kl, new, scale=c.scale)
    ref.check_attention(out.double().cpu().numpy(), None, c.want(), D, 150)


def test_large_scores(sv):
    """Scores of some thousands: every weight but the largest underflows."""
    c = Case(64, 2, 1, 16, [80], [2], seed=10, spread=300.0)
    c.check(sv)


def _dense(q, k, v, table, page, ctx, n, scale):
    """One request in float64 on the device: out, lse."""
    Hq, D = q.shape[1:]
    Hkv = k.shape[1]
    held = table[0, :-(-(ctx + n) // page)].long()
    kk, vv = (t[held].transpose(0, 1).reshape(Hkv, -1, D)[:, :ctx + n].double() for t in (k, v))
    x = torch.einsum("tgd,gjd->gtj", q.double(), kk.repeat_interleave(Hq // Hkv, 0)) * scale
    at = torch.arange(ctx + n, device=q.device)
    x = x.masked_fill(at[None, None, :] > ctx + torch.arange(n, device=q.device)[None, :, None],
                      -math.inf)
    out = torch.einsum("gtj,gjd->tgd", x.softmax(-1), vv.repeat_interleave(Hq // Hkv, 0))
    return out, x.logsumexp(-1).T


@pytest.mark.parametrize("D,n,ctx,Hq,Hkv,page", [
    (64, 600, 9000, 4, 1, 16), (128, 600, 9000, 4, 1, 64), (256, 600, 9000, 4, 1, 16),
    (256, 300, 20000, 2, 2, 128), (128, 2000, 0, 10, 2, 16), (256, 2000, 0, 10, 2, 32),
    (256, 70, 40000, 1, 1, 64), (128, 70, 40000, 1, 1, 64)])
def test_long_chunks(sv, D, n, ctx, Hq, Hkv, page):
    """Segments of many tiles, where a wait on a wrong phase shows: no wait may
    give up, and every run gives the same bits."""
    d = dev()
    g = torch.Generator(device=d)
    g.manual_seed(n + ctx + D)
    held = -(-(ctx + n) // page)
    k, v = (torch.randn(held, Hkv, page, D, generator=g, device=d, dtype=torch.bfloat16)
            for _ in range(2))
    q = torch.randn(n, Hq, D, generator=g, device=d, dtype=torch.bfloat16) * 1.5
    table = torch.randperm(held, generator=g, device=d).to(torch.int32)[None].contiguous()
    qs = torch.tensor([0, n], dtype=torch.int32, device=d)
    kl = torch.tensor([ctx + n], dtype=torch.int32, device=d)
    lse = torch.empty(n, Hq, device=d)
    ws = sv.make_attention_workspace(D, d)
    scale = 1.0 / math.sqrt(D)
    out = sv.paged_attention(q, k, v, table, qs, kl, n, lse=lse, workspace=ws)[0].clone()
    sv.device_status()
    for _ in range(10):
        assert torch.equal(sv.paged_attention(q, k, v, table, qs, kl, n, workspace=ws)[0], out)
    sv.device_status()
    want, want_lse = _dense(q, k, v, table, page, ctx, n, scale)
    # weights and outputs are rounded to bf16 (2^-8 at most each, in norm as well)
    assert float((out.double() - want).norm() / want.norm()) < 2 * ref.HALF_BF16
    # scores of magnitude 10: D fp32 sums, the exponential's 2^-21, 20000 sums
    assert float((lse.double() - want_lse).abs().max()) < 10 * (D + 4) * 2.0 ** -24 + 2.0 ** -9


@pytest.mark.parametrize("D,most", [(64, 2), (128, 2), (256, 1), (64, 40), (128, 40), (256, 40)])
def test_more_requests_than_threads(sv, D, most):
    """The search for a CTA's first request goes on in the next block of them."""
    rng = np.random.default_rng(D + most)
    B = 900
    lens = rng.integers(0, 60, B).tolist()
    news = [int(min(n, rng.integers(0, most + 1))) for n in lens]
    lens[500], news[500] = 700, most
    Case(D, 2, 1, 16, lens, news, seed=most).check(sv, max_new=100 if most > 2 else None)


@pytest.mark.parametrize("D,news", [(64, [7, 3]), (128, [90, 3]), (256, [90, 7])])
def test_the_widest_window_is_none(sv, D, news):
    c = Case(D, 4, 2, 16, [40, 5], news, seed=11)
    c.check(sv, 2 ** 31 - 1)
    c.check(sv, 45)
