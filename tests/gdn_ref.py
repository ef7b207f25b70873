"""Plain references of the GatedDeltaNet operators over packed rows for their
parity tests: each follows the definition in include/specverify.h row by row, in
float64 on the host, sharing no code with the kernels."""
import numpy as np

HALF_BF16 = 2.0 ** -8   # a rounding to nearest is off by at most half a step,
HALF_F32 = 2.0 ** -24   # relative to the value


def _spans(q_start, rows):
    s = np.clip(np.asarray(q_start, np.int64), 0, rows)
    return [(int(s[b]), int(max(s[b + 1], s[b]))) for b in range(len(s) - 1)]


def inputs(x, a, b, weight, window, a_log, dt_bias, q_start, k_heads, dk, index=None, update=True,
           q_scale=1.0, eps=1e-6):
    """gdn_inputs.  Returns (q, k, v, alpha, beta, window) and, for the bounds,
    the magnitude of the terms of every output."""
    x, a, b, weight, window, a_log, dt_bias = (np.asarray(t, np.float64) for t in
                                               (x, a, b, weight, window, a_log, dt_bias))
    rows, C = x.shape
    W, H = weight.shape[0], a.shape[1]
    Hk, dv = k_heads, (C - 2 * k_heads * dk) // H
    y, mag = np.zeros((rows, C)), np.zeros((rows, C))
    alpha, beta = np.zeros((rows, H)), np.zeros((rows, H))
    window, slots = window.copy(), window.shape[0]
    real = np.zeros(rows, bool)
    for s, (r0, r1) in enumerate(_spans(q_start, rows)):
        slot = s if index is None else int(index[s])
        if r1 == r0 or not 0 <= slot < slots:
            continue
        real[r0:r1] = True
        past = np.concatenate([window[slot], x[r0:r1]])
        for t in range(r1 - r0):
            y[r0 + t] = (weight * past[t:t + W]).sum(0)
            mag[r0 + t] = np.abs(weight * past[t:t + W]).sum(0)
        if update:
            window[slot] = past[r1 - r0:]
    with np.errstate(over="ignore"):
        y = y / (1 + np.exp(-y))
        alpha = np.exp(-np.exp(a_log) * np.logaddexp(a + dt_bias, 0)) * real[:, None]
        beta = 1 / (1 + np.exp(-b)) * real[:, None]
    q, k = (y[:, i * Hk * dk:(i + 1) * Hk * dk].reshape(rows, Hk, dk) for i in (0, 1))
    v = y[:, 2 * Hk * dk:].reshape(rows, H, dv)
    norm = [np.sqrt((t * t).sum(-1, keepdims=True) + eps) for t in (q, k)]
    f = [q_scale / norm[0], 1 / norm[1]]
    mags = [mag[:, i * Hk * dk:(i + 1) * Hk * dk].reshape(rows, Hk, dk) for i in (0, 1)]
    # a head's outputs also carry its norm's error, at most that of its terms
    spread = [np.abs(f[i]) * (mags[i] + np.sqrt((mags[i] ** 2).sum(-1, keepdims=True))
                              * np.abs((q, k)[i]) / norm[i]) for i in (0, 1)]
    return ((q * f[0], k * f[1], v, alpha, beta, window),
            (spread[0], spread[1], mag[:, 2 * Hk * dk:].reshape(rows, H, dv)))


def advance(q, k, v, alpha, beta, state, q_start, index=None, chunk=1, tol=0.0):
    """gdn_advance, token by token.  Returns out, state and bounds for them: of
    each output, and of each row of the state in norm.

    A step maps a row s of S to alpha s (1 - beta k k^T) + beta v k^T, which
    shrinks any error in s while beta |k|^2 <= 2, so the errors of the steps add
    up, each decayed by the gates after it.  A step's own: the decayed row, the
    dot product with k, e and the rank-1 term are each rounded a few times, and
    in chunks e is a sum over the rows e_j before it in the chunk, with factors
    of norm at most 1.  Roundings are independent, so n of them count sqrt(n):
    with dk + chunk <= 256 terms and 6 operations on each at most 40 half steps
    of (|s| + |v| + |e of the last rows|) |k|.

    Of bf16 rows in chunks the output takes the chunk's first state, every e_j and
    their factors in two bf16 parts each, cut off: 2^-15 of the value is left out, and
    the product of two second parts, below 2^-14 of theirs."""
    q, k, v, alpha, beta = (np.asarray(t, np.float64) for t in (q, k, v, alpha, beta))
    state = np.asarray(state, np.float64).copy()
    rows, Hk, dk = q.shape
    slots, H, dv, _ = state.shape
    G = H // Hk
    out, out_tol = np.zeros((rows, H, dv)), np.zeros((rows, H, dv))
    tol = np.zeros((slots, H, dv)) + tol  # the state's own error before
    u = 40 * HALF_F32
    for s, (r0, r1) in enumerate(_spans(q_start, rows)):
        slot = s if index is None else int(index[s])
        if not 0 <= slot < slots:
            continue
        S, err = state[slot], tol[slot]
        for r in range(r0, r1):
            if (r - r0) % chunk == 0:  # the chunk's rows so far, their gates, its first state
                past_e, past_k, gates = [], [], []
                first, g0 = np.linalg.norm(S, axis=-1), np.ones(H)
            kk, qq = np.repeat(k[r], G, 0), np.repeat(q[r], G, 0)
            S *= alpha[r][:, None, None]
            size = np.linalg.norm(S, axis=-1)
            e = beta[r][:, None] * (v[r] - np.einsum("hij,hj->hi", S, kk))
            S += e[..., None] * kk[:, None]
            out[r] = np.einsum("hij,hj->hi", S, qq)
            gates = [g * alpha[r] for g in gates] + [np.ones(H)]
            g0 = g0 * alpha[r]
            past_e.append(np.abs(e))
            past_k.append(kk)
            kn, qn = (np.linalg.norm(t, axis=-1)[:, None] for t in (kk, qq))
            near = np.sqrt((np.array(past_e) ** 2).sum(0))
            err[:] = err * alpha[r][:, None] + u * (size + (np.abs(v[r]) + near) * kn)
            out_tol[r] = err * qn + u * (np.linalg.norm(S, axis=-1) + near * kn) * qn
            if chunk > 1:
                factors = np.abs(np.einsum("jhd,hd->jh", np.array(past_k), qq)) * np.array(gates)
                terms = np.einsum("jh,jhi->hi", factors, np.array(past_e))
                out_tol[r] += 2.0 ** -13 * terms + 2.0 ** -15 * first * g0[:, None] * qn
    return out, state, out_tol, tol
