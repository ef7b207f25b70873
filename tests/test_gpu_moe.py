"""moe_smallm against float64."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import dev, sv_module

pytestmark = pytest.mark.gpu
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    return sv_module()


class Layer:
    def __init__(self, rows, hidden, inter, experts, top, seed=0):
        self.sizes = rows, hidden, inter, experts, top
        g = torch.Generator(device=dev())
        g.manual_seed(seed)

        def four_bit(n, k):
            words = torch.randint(-2**31, 2**31, (experts, n, k // 8), generator=g, device=dev(),
                                  dtype=torch.int64).to(torch.int32)
            s = (torch.rand(experts, n, k // 64, generator=g, device=dev()) + 0.5) / (4.6 * k ** 0.5)
            return words, s.bfloat16(), (s * -7.5 + 0.01).bfloat16()

        rand = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
        self.x = rand(rows, hidden).bfloat16()
        self.router = (rand(experts, hidden) / hidden ** 0.5).bfloat16()
        self.gate, self.up, self.down = four_bit(inter, hidden), four_bit(inter, hidden), four_bit(hidden, inter)
        self.ids = torch.full((rows, top), -1, dtype=torch.int32, device=dev())
        self.weights = torch.full((rows, top), -1.0, device=dev())

    def run(self, sv, **kw):
        return sv.moe_smallm(self.x, self.router, self.gate, self.up, self.down, self.sizes[4],
                             ids=self.ids, weights=self.weights, **kw)

    def want(self, **kw):
        host = lambda m: [m[0].cpu().numpy(), m[1].double().cpu().numpy(), m[2].double().cpu().numpy()]  # noqa: E731
        return ref.layer(self.x.double().cpu().numpy(), self.router.double().cpu().numpy(),
                         host(self.gate), host(self.up), host(self.down), self.sizes[4], **kw)


def _check(layer, y, **kw):
    hidden, inter = layer.sizes[1:3]
    ids = layer.ids.cpu().numpy()
    y_want, _, w, mag, z, terms = layer.want(ids=ids, **kw)
    # the logits are fp32 sums of `hidden` products (independent roundings: their root):
    # in the order of choice they fall, and none left out is above the last
    tol = 4 * hidden ** 0.5 * HALF_F32 * terms.max()
    chosen = np.take_along_axis(z, ids, 1)
    assert (np.diff(chosen, axis=1) <= tol).all()
    left = z.copy()
    np.put_along_axis(left, ids, -np.inf, 1)
    assert (left.max(1) <= chosen[:, -1] + tol).all()
    got = layer.weights.double().cpu().numpy()
    assert (np.abs(got - w) <= (2 * tol + 64 * HALF_F32) * w + 1e-30).all()
    # fp32 sums of `hidden` and `inter` products, each group's offset of 128 times its
    # inputs' sum (8 bits of the fp32 products' place), the activations as two bf16
    # parts (2^-16), y rounded to bf16
    u = 2.0 ** -16 + (hidden + inter) ** 0.5 * 2 ** 8 * HALF_F32
    bound = (HALF_BF16 + 2 * tol) * np.abs(y_want) + u * mag
    err = np.abs(y.double().cpu().numpy() - y_want)
    assert (err <= bound).all()


@pytest.mark.parametrize("rows,hidden,inter,experts,top", [
    (1, 128, 128, 1, 1), (1, 256, 128, 4, 2), (1, 2048, 512, 256, 8), (2, 512, 256, 8, 8),
    (4, 1280, 384, 64, 6), (8, 384, 896, 12, 3), (9, 256, 256, 3, 1), (17, 640, 128, 60, 4),
    (33, 512, 384, 5, 2), (64, 128, 640, 100, 16), (128, 1024, 256, 32, 4), (128, 256, 128, 2, 2),
    (100, 256, 128, 512, 7), (3, 2560, 1024, 40, 5)])
def test_layer(sv, rows, hidden, inter, experts, top):
    c = Layer(rows, hidden, inter, experts, top, seed=rows + hidden)
    _check(c, c.run(sv))
    sv.device_status()


def test_softmax_over_all_experts(sv):
    c = Layer(5, 256, 128, 16, 4, seed=1)
    _check(c, c.run(sv, renormalize=False), renormalize=False)


def test_equal_logits_take_the_lower_expert(sv):
    """The same router row for several experts, and one row of zeros of x."""
    c = Layer(4, 256, 128, 24, 5, seed=2)
    c.router[7] = c.router[3]
    c.router[20] = c.router[3]
    c.x[2] = 0.0
    c.run(sv)
    z = c.x.double() @ c.router.double().T
    for t in range(4):
        best = sorted(range(24), key=lambda e: (-float(z[t, e]), e))[:5]
        assert c.ids[t].tolist() == best
    assert c.ids[2].tolist() == [0, 1, 2, 3, 4]


def test_one_expert_takes_every_row(sv):
    """Slots of one expert: 128 rows of it, in slots of 8."""
    c = Layer(128, 256, 256, 8, 1, seed=3)
    c.x = c.x.abs()
    c.router[:] = -1.0
    c.router[5] = 1.0
    _check(c, c.run(sv))
    assert (c.ids == 5).all()


def test_rows_that_are_not_finite_keep_to_themselves(sv):
    c = Layer(6, 256, 128, 16, 3, seed=4)
    clean = c.run(sv).clone()
    c.x[1, 5] = float("nan")
    c.x[4, 200] = float("inf")
    y = c.run(sv)
    keep = [0, 2, 3, 5]
    assert y[1].isnan().all() and not y[4].isfinite().all()
    assert c.ids[1].tolist() == [0, 1, 2]  # no order among NaN but the index
    # the others' sums may be cut elsewhere: near, not equal
    scale = clean[keep].float().norm(dim=1)
    assert ((y[keep].float() - clean[keep].float()).norm(dim=1) <= 2 * HALF_BF16 * scale).all()


def test_the_same_bits_again_in_a_graph_and_on_two_streams(sv):
    c = Layer(12, 512, 384, 30, 4, seed=5)
    sizes = c.sizes
    ws = sv.make_moe_workspace(*sizes, dev())
    want = c.run(sv, workspace=ws).clone()
    for _ in range(20):
        assert torch.equal(c.run(sv, workspace=ws), want)
    sides = [(torch.cuda.Stream(), sv.make_moe_workspace(*sizes, dev()), torch.empty_like(want))
             for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, w, out in sides:
            with torch.cuda.stream(stream):
                sv.moe_smallm(c.x, c.router, c.gate, c.up, c.down, sizes[4], out=out, workspace=w)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, _, out in sides)
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(sv, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    n, zero = sv.moe_smallm_workspace_bytes(*sizes)
    assert ws.numel() == n and not ws[:zero].any()
    sv.set_pdl(True)
    try:
        assert all(torch.equal(c.run(sv, workspace=ws), want) for _ in range(10))
    finally:
        sv.set_pdl(False)
    sv.device_status()


def test_no_rows(sv):
    c = Layer(0, 256, 128, 4, 2, seed=6)
    assert c.run(sv).shape == (0, 256)
