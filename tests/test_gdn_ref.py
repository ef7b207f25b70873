"""The GatedDeltaNet references for packed rows against the oracle's capture and
convolution (CPU)."""
import numpy as np
import pytest

import gdn_ref as ref
import workloads as wl


@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (3, 5, 2), (2, 16, 3)])
def test_advance_reference_is_the_tapes_recurrence(oracle, B, T, H):
    g = wl.gdn_inputs(1, B, T, H, 24, 16)
    want, tape = oracle.gdn_capture(g["state0"], g["q"], g["k"], g["v"], g["alpha"], g["beta"])
    flat = {n: g[n].reshape(B * T, *g[n].shape[2:]) for n in ("q", "k", "v", "alpha", "beta")}
    out, state, _, _ = ref.advance(**flat, state=g["state0"], q_start=np.arange(B + 1) * T)
    assert np.abs(out.reshape(B, T, H, 16) - want).max() < 1e-6
    all_of = oracle.gdn_replay(g["state0"], tape, np.full(B, T, np.int32))
    assert np.abs(state - all_of).max() < 1e-6


def test_advance_reference_shares_heads_and_follows_the_slots():
    r = np.random.default_rng(0)
    q, k = r.normal(size=(5, 2, 8)), r.normal(size=(5, 2, 8)) / 8
    v, al, be = r.normal(size=(5, 4, 8)), r.random((5, 4)), r.random((5, 4))
    state = r.normal(size=(3, 4, 8, 8))
    out, new, _, _ = ref.advance(q, k, v, al, be, state, [0, 2, 2, 4], index=[2, 0, 9])
    one, S, _, _ = ref.advance(q[:2, 1:], k[:2, 1:], v[:2, 2:], al[:2, 2:], be[:2, 2:],
                               state[2:, 2:], [0, 2])
    assert np.array_equal(out[:2, 2:], one) and np.array_equal(new[2:, 2:], S)
    assert np.array_equal(new[:2], state[:2]) and (out[2:] == 0).all()


@pytest.mark.parametrize("W,n", [(4, 1), (4, 2), (4, 7), (2, 1), (8, 3)])
def test_inputs_reference_is_the_window_convolution(oracle, W, n):
    c = wl.conv_inputs(2, 1, n, 2 * 8 + 3 * 8, W)
    x = c["x"][0].astype(np.float64)
    y = oracle.conv_capture(c["window"], c["x"], c["weight"])[0].astype(np.float64)
    gates = np.random.default_rng(1).normal(size=(2, n, 3))
    (q, k, v, al, be, win), _ = ref.inputs(x, *gates, c["weight"], c["window"], np.zeros(3),
                                           np.ones(3), [0, n], 1, 8, q_scale=0.5)
    y = y / (1 + np.exp(-y))
    assert np.abs(v.reshape(n, -1) - y[:, 16:]).max() < 1e-6
    for got, want, scale in ((q, y[:, :8], 0.5), (k, y[:, 8:16], 1.0)):
        assert np.abs(got[:, 0] - scale * want / np.sqrt((want ** 2).sum(-1, keepdims=True) + 1e-6)).max() < 1e-5
    assert np.abs(al - (1 + np.exp(gates[0] + 1)) ** -1.0).max() < 1e-12
    assert np.abs(be - 1 / (1 + np.exp(-gates[1]))).max() < 1e-12
    want = oracle.conv_replay(c["window"], c["x"], np.array([n], np.int32))
    assert np.array_equal(win, want.astype(np.float64))
