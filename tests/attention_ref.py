"""Plain references of the paged-cache operators for their parity tests: each
follows the definition in include/specverify.h step by step, in float64 (or
Python integers) on the host, sharing no code with the kernels."""
import math

import numpy as np


def pages_step(length, held, cursor, ring, table, n_new, page, rows, commit=None, bias=0):
    """kv_pages_step, one request after another.  Returns a dict of the outputs."""
    B, max_pages = table.shape
    P = len(ring)
    ring0, ring, table = ring.copy(), ring.copy(), table.copy()
    flags0 = 0
    head, free = int(cursor[0]), int(cursor[1])
    if not 0 <= head < P or not 0 <= free <= P:
        flags0 = 128
    head, free = min(max(head, 0), P - 1), min(max(free, 0), P)
    out = {k: np.zeros(B, np.int32) for k in ("length", "held", "kv_len", "err_flags")}
    out["q_start"] = np.zeros(B + 1, np.int32)
    out["slots"] = np.full(rows, -1, np.int32)
    out["positions"] = np.zeros(rows, np.int32)
    row = asked = used = 0
    back = []
    givers = []
    for b in range(B):
        fl = flags0
        h = min(max(int(held[b]), 0), max_pages)
        if h != held[b]:
            fl |= 128
        n = int(n_new[b])
        grown = int(length[b]) + (int(commit[b % len(commit)]) + bias if commit is not None else 0)
        L = min(max(grown, 0), h * page)
        ended = n < 0
        if ended:
            L, n = 0, 0
            back += [int(x) for x in table[b, :h]]
            givers += [b] * h
        elif L != grown:
            fl |= 16
        refused = False
        got = 0
        if n > 0 and row + n > rows:
            refused, fl = True, fl | 64
        want = -(-(L + n) // page)
        if want > max_pages:
            refused, fl = True, fl | 32
        if not refused and not ended:
            need = max(0, want - h)
            if need and asked + need > free:
                refused, fl = True, fl | 32
            else:
                got = need
            asked += need
        for i in range(got):
            table[b, h + i] = ring0[(head + used + i) % P]
        used += got
        out["length"][b] = L
        out["held"][b] = 0 if ended else h + got
        out["kv_len"][b] = 0 if refused else L + n
        out["err_flags"][b] = fl
        out["q_start"][b] = min(row, rows)
        for t in range(n):
            r = row + t
            if r < rows:
                out["positions"][r] = L + t
                if not refused:
                    pg = int(table[b, (L + t) // page])
                    if 0 <= pg < P:
                        out["slots"][r] = pg * page + (L + t) % page
        row += n
    out["q_start"][B] = min(row, rows)
    room = P - free
    for i, pg in enumerate(back[:room]):
        ring[(head + free + i) % P] = pg
    if len(back) > room:
        for b in set(givers) | {b for b in range(B) if n_new[b] < 0}:
            out["err_flags"][b] |= 128
    out["cursor"] = np.array([(head + used) % P, free - used + min(len(back), room)], np.int32)
    out["block_table"], out["ring"] = table, ring
    return out


def rotate(x, positions, inv_freq, axis=None, weight=None, eps=1e-6, interleaved=False):
    """Norm and rotary positions of x [rows, heads, D] (float64); also returns
    the bound's scale: the magnitude of the two terms of every element."""
    x = np.asarray(x, np.float64)
    rows, heads, D = x.shape
    y = x.copy()
    if weight is not None:
        y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out, mag = y.copy(), np.abs(y)
    half = len(inv_freq)
    pos = positions.reshape(rows, -1).astype(np.float64)
    for f in range(half):
        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        t = pos[:, int(axis[f]) if axis is not None else 0] * inv_freq[f]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = np.abs(y[:, :, a]) + np.abs(y[:, :, b])
    return out, mag


def attention(q, k_cache, v_cache, table, q_start, kv_len, scale, window=0):
    """paged_attention row by row.  Returns out, lse and, for the bounds, the
    weighted magnitude of the values [rows, Hq, D] and the largest magnitude of
    a score's products [rows, Hq]."""
    rows, Hq, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out = np.zeros((rows, Hq, D))
    lse = np.full((rows, Hq), -np.inf)
    mag = np.zeros((rows, Hq, D))
    smag = np.zeros((rows, Hq))
    for b in range(len(kv_len)):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        for r in range(r0, r1):
            p = int(kv_len[b]) - (r1 - r0) + (r - r0)
            j = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            if len(j) == 0:
                continue
            pg = table[b, j // page]
            ok = (pg >= 0) & (pg < pages)
            pg = np.where(ok, pg, 0)
            for h in range(Hkv):
                k = np.where(ok[:, None], k_cache[pg, h, j % page], 0.0).astype(np.float64)
                v = np.where(ok[:, None], v_cache[pg, h, j % page], 0.0).astype(np.float64)
                for g in range(G):
                    x = q[r, h * G + g].astype(np.float64)
                    s = k @ x * scale
                    m = s.max()
                    w = np.exp(s - m)
                    total = w.sum()
                    out[r, h * G + g] = (w / total) @ v
                    lse[r, h * G + g] = m + math.log(total) if np.isfinite(total) else np.nan
                    mag[r, h * G + g] = (w / total) @ np.abs(v)
                    smag[r, h * G + g] = scale * (np.abs(k) @ np.abs(x)).max()
    return out, lse, mag, smag


HALF_BF16 = 2.0 ** -8  # a bf16 rounding, relative to the value


def check_attention(out, lse, ref, D, keys):
    """Bounds for `keys` attended at most.  A score sums D exact products in
    fp32, is scaled and goes through a base-2 exponential, each off by at most
    d = ((D + 4) 2^-24) smag + 2^-21 in the exponent; the weight is rounded to
    bf16, the sums of the weights and of the products carry keys + 8 fp32
    additions (splits and joins rescale a few times), and the output is
    rounded to bf16."""
    want, want_lse, mag, smag = ref
    d = (D + 4) * 2.0 ** -24 * smag + 2.0 ** -21
    acc = (keys + 8) * 2.0 ** -24
    tol = HALF_BF16 * np.abs(want) + (HALF_BF16 + 2 * (d[..., None] + acc)) * (1 + HALF_BF16) * mag
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(out), nan)
    err = np.where(nan, 0.0, np.abs(out - want))
    bad = err > np.where(nan, 1.0, tol) + 1e-30
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside; first {np.argwhere(bad)[:3].tolist()}"
                           f" got {out[bad][:3]} want {want[bad][:3]} tol {tol[bad][:3]}")
    if lse is not None:
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(lse), none)
        fin = np.isfinite(want_lse)
        assert np.array_equal(np.isnan(lse), ~fin & ~none)
        tl = d + acc + 2.0 ** -21 + np.abs(np.where(fin, want_lse, 0)) * 2.0 ** -22
        e = np.where(fin, np.abs(np.where(fin, lse, 0) - np.where(fin, want_lse, 0)), 0)
        assert (e <= tl).all(), (e.max(), tl[np.unravel_index(e.argmax(), e.shape)])
