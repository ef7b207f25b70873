"""moe_smallm in float64, and how far off fp32 arithmetic may leave its outputs before
their one rounding: the independent roundings of each sum, added as such.

With h = 2^-24, a half step.  A group of 64 products is four steps of 16 on the tensor
cores, each cut off by half a last place on average, a half step of the sum so far at most;
the inputs' sum for the bias is six roundings; then each group adds two roundings to the
running sum.  A sum so far, of terms of either sign, is about the root of the sum of its
terms' squares, the nibbles' s q x and the biases' b x apart.  So a sum over n groups is
off by h sqrt(4^2 + 8 + 2 n) of that root.  silu's derivative is at most 1.1; an
exponential, a division and two products are 8 half steps; the activations in two fp16
parts are off by 2^-24 of their group's largest.  A weight is off by twice its logits'
error (steps of 16 over 16 warps, then the warps) and 8 half steps."""
import numpy as np

from moe_ref import choose

H = 2.0 ** -24


def parts(words, scales, biases):
    """The nibbles' and the biases' parts of a matrix [N, K] apart, in float64."""
    words = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    q = np.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).reshape(words.shape[0], -1)
    wide = [np.repeat(np.asarray(t, np.float64), 64, 1) for t in (scales, biases)]
    return q * wide[0], wide[1]


def _sum(matrix, x):
    """A product with each of the rows x [n, K]: the values, and their error's root."""
    a, b = matrix
    squares = x ** 2 @ (a ** 2 + b ** 2).T
    return x @ (a + b).T, H * np.sqrt((24 + 2 * (a.shape[1] / 64)) * squares)


def layer(x, router, gate, up, down, top, renormalize=True, ids=None):
    """y, its error before the rounding, and the experts: as given, or its own choice."""
    x, router = np.asarray(x, np.float64), np.asarray(router, np.float64)
    rows, hidden = x.shape
    z = x @ router.T
    if ids is None:
        ids = np.array([choose(r, top) for r in z], np.int32).reshape(rows, top)
    best = np.take_along_axis(z, ids, 1)
    w = np.exp(best - best[:, :1])
    w /= (w if renormalize else np.exp(z - best[:, :1])).sum(1, keepdims=True)
    err_z = (16 + hidden / 256) * H * np.sqrt((x ** 2 @ router.T ** 2).max(1))
    y, square = np.zeros((rows, hidden)), np.zeros((rows, hidden))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        G, U, D = (parts(*(m[e] for m in w3)) for w3 in (gate, up, down))
        (g, err_g), (u, err_u) = _sum(G, x[t]), _sum(U, x[t])
        silu = g / (1 + np.exp(-g))
        h = silu * u
        most = np.repeat(np.abs(h).reshape(len(t), -1, 64).max(-1), 64, 1)
        err_h = np.sqrt((1.1 * u * err_g) ** 2 + (silu * err_u) ** 2 + (8 * H * h) ** 2 + (H * most) ** 2)
        out, err = _sum(D, h)
        share = w[t, j][:, None]
        y[t] += share * out
        square[t] += share ** 2 * (err_h ** 2 @ ((D[0] + D[1]) ** 2).T + err ** 2
                                   + ((2 * err_z[t][:, None] + 12 * H) * out) ** 2)
    return y, np.sqrt(square), ids
