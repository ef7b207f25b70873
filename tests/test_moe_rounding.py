"""What the check of moe_smallm's outputs finds and what it passes (CPU): the layer made
wrong, or in fewer bits, in each of the ways that a kernel may be."""
import numpy as np
import pytest

import moe_rounding as ref
import rounding


def _bf16(v):
    return rounding.nearest(v)


def _layer(rows, hidden, inter, experts, top, seed):
    r = np.random.default_rng(seed)

    def four_bit(n, k):
        s = (r.random((experts, n, k // 64)) + 0.5) / (4.6 * k ** 0.5)
        return (r.integers(0, 2 ** 32, (experts, n, k // 8)), _bf16(s), _bf16(s * -7.5 + 0.01))

    return (_bf16(r.normal(size=(rows, hidden))), _bf16(r.normal(size=(experts, hidden)) / hidden ** 0.5),
            four_bit(inter, hidden), four_bit(inter, hidden), four_bit(hidden, inter), top)


def _fp16(v, parts):
    """Rows of activations in fp16 parts, a power of two for each group of 64."""
    g = v.reshape(len(v), -1, 64)
    scale = 2.0 ** (14 - np.floor(np.log2(np.abs(g).max(-1, keepdims=True))))
    rest, out = g * scale, 0.0
    for _ in range(parts):
        part = rest.astype(np.float16).astype(np.float64)
        out, rest = out + part, rest - part
    return (out / scale).reshape(v.shape)


def _computed(args, offset=0.0, act_parts=2, lose=None):
    """The layer as the kernel computes it, sums in fp32, and with one thing wrong."""
    x, router, gate, up, down, top = args
    _, _, ids = ref.layer(*args)
    z = x @ router.T
    w = np.exp(np.take_along_axis(z, ids, 1))
    w /= w.sum(1, keepdims=True)
    y = np.zeros(x.shape)

    def product(m, v, e, gone=None):
        words, s, b = (t[e] for t in m)
        q = np.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).reshape(words.shape[0], -1)
        if lose == "a low bit of every eighth nibble":
            q[:, ::8] &= 14
        total = np.zeros((len(v), len(q)), np.float32)
        for g in range(q.shape[1] // 64):
            at = slice(64 * g, 64 * g + 64)
            if g == gone:
                continue
            d = np.repeat((-offset * v[:, at].sum(1))[:, None], len(q), 1).astype(np.float32)
            for k in range(64 * g, 64 * g + 64, 16):
                d = (d + v[:, k:k + 16] @ (q[:, k:k + 16] + offset).T).astype(np.float32)
            bias = (b[:, g] * v[:, at].sum(1)[:, None].astype(np.float32)).astype(np.float64)
            total = (s[:, g] * d + (bias + total).astype(np.float32)).astype(np.float32)
        return total.astype(np.float64)

    for j in range(top - (lose == "the last expert")):
        for e in np.unique(ids[:, j]):
            t = np.nonzero(ids[:, j] == e)[0]
            g = product(gate, x[t], e, 1 if lose == "a group of gate" else None)
            u = product(up, x[t], e)
            h = _fp16((g / (1 + np.exp(-g)) * u).astype(np.float32).astype(np.float64), act_parts)
            y[t] += w[t, j][:, None] * product(down, h, e)
    return _bf16((y * (1.05 if lose == "a factor of 1.05" else 1.0)).astype(np.float32).astype(np.float64))


SIZES = [(1, 2048, 512, 8, 8), (8, 2560, 1024, 4, 2), (16, 1024, 256, 4, 2)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_passes_fp32_sums(sizes):
    args = _layer(*sizes, seed=1)
    want, err, _ = ref.layer(*args)
    assert rounding.faults(_computed(args), want, err) is None


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("lose", ["the last expert", "a group of gate", "a factor of 1.05",
                                  "a low bit of every eighth nibble"])
def test_finds_what_is_left_out(sizes, lose):
    args = _layer(*sizes, seed=1)
    want, err, _ = ref.layer(*args)
    assert rounding.faults(_computed(args, lose=lose), want, err) is not None


@pytest.mark.parametrize("kw", [{"act_parts": 1}, {"offset": 1024.0}], ids=str)
def test_finds_fewer_bits(kw):
    args = _layer(48, 1024, 512, 4, 2, seed=2)
    want, err, _ = ref.layer(*args)
    assert rounding.faults(_computed(args), want, err) is None
    assert rounding.faults(_computed(args, **kw), want, err) is not None
