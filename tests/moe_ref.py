"""A plain reference of moe_smallm in float64 on the host, step by step from the
definition in include/specverify.h, sharing no code with the kernels."""
import numpy as np


def dequantise(words, scales, biases):
    """w_packed uint32 [N, K/8], scales, biases [N, K/64] -> W float64 [N, K]."""
    words = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    q = np.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).reshape(words.shape[0], -1)
    return q * np.repeat(np.asarray(scales, np.float64), 64, 1) + \
        np.repeat(np.asarray(biases, np.float64), 64, 1)


def choose(z, top):
    """The top largest of a row of logits: equal ones by the lower index, NaN last."""
    key = [(np.isnan(v), -v if not np.isnan(v) else 0.0, e) for e, v in enumerate(z)]
    return [k[2] for k in sorted(key)[:top]]


def layer(x, router, gate, up, down, top, renormalize=True, ids=None):
    """Returns y, ids, weights, the magnitude of y's terms for the bounds, the logits
    and the magnitude of their terms; with the given choice, or its own."""
    x, router = np.asarray(x, np.float64), np.asarray(router, np.float64)
    rows, hidden = x.shape
    z = x @ router.T
    if ids is None:
        ids = np.array([choose(r, top) for r in z], np.int32).reshape(rows, top)
    with np.errstate(invalid="ignore"):
        w = np.exp(z[np.arange(rows)[:, None], ids] - z[np.arange(rows), ids[:, 0]][:, None])
        rest = w.sum(1) if renormalize else np.exp(z - z[np.arange(rows), ids[:, 0]][:, None]).sum(1)
    w = w / rest[:, None]
    y, mag = np.zeros((rows, hidden)), np.zeros((rows, hidden))
    for e in np.unique(ids):
        G, U, D = (dequantise(*(t[e] for t in m)) for m in (gate, up, down))
        for t, j in np.argwhere(ids == e):
            g, u = G @ x[t], U @ x[t]
            h = g / (1 + np.exp(-g)) * u
            y[t] += w[t, j] * (D @ h)
            # an error of h in proportion to its factors' terms, then down's terms
            hm = (np.abs(G) @ np.abs(x[t])) * np.abs(u) + np.abs(g) * (np.abs(U) @ np.abs(x[t]))
            mag[t] += w[t, j] * (np.abs(D) @ (np.abs(h) + hm))
    return y, ids, w, mag, z, np.abs(x) @ np.abs(router).T
