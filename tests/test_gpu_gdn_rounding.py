"""gdn_advance's bf16 outputs are fp32 results rounded once, row after row and in chunks."""
import numpy as np
import pytest
import torch

import gdn_ref as ref
import rounding
from gpu_util import sv_module
from test_gpu_gdn_rows import Rows, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def _outputs(q, k, v, alpha, beta, state):
    """One sequence of at most 64 rows: its outputs in float64, and how far off fp32
    arithmetic may leave them before the rounding.

    With D the gates from a row to the next ones and G those from the first, a row is
        e = beta (v - G S0 k - sum D (k . k_j) e_j),   o = G S0 q + sum D (q . k_j) e_j.
    On the tensor cores a sum is cut off at each step of 16 terms, by half a last place on
    average: one half step (2^-24) of the sum so far at most.  The full-sized steps are 8
    of S0 k or S0 q (128 terms) and 4 of each triangle (64 rows): V T^T and R T^T for e,
    E P^T for o; T is off by 2^-22 of its terms on average.  That makes 8 + 4 + 4 + 4 = 20
    half steps for e and, with the sum of both parts, 8 + 4 + 1 = 13 for o.  A sum so
    far, of terms of either sign, is about the root of the sum of its terms' squares.
    Row after row there are fewer steps and they are rounded.  The errors of the e_j
    reach o with the e_j's factors."""
    rows, H, dv = v.shape
    G = H // q.shape[1]
    q, k = np.repeat(q, G, 1), np.repeat(k, G, 1)
    out, err = np.zeros(v.shape), np.zeros(v.shape)
    e, err_e = np.zeros(v.shape), np.zeros(v.shape)
    g = np.ones(H)
    decay = np.zeros((0, H))  # D of the rows so far
    for r in range(rows):
        g = g * alpha[r]
        decay = np.concatenate([decay * alpha[r], np.ones((1, H))])

        def sums(x, upto):
            """S0 x + sum over rows < upto of D (k_j . x) e_j: the sum, the sum of its
            terms' squares, and that of the e_j's errors."""
            f = decay[:upto] * np.einsum("jhd,hd->jh", k[:upto], x)
            near = f[..., None] * e[:upto]
            far = g[:, None, None] * state * x[:, None]
            return (far.sum(-1) + near.sum(0), (far ** 2).sum(-1) + (near ** 2).sum(0),
                    ((f[..., None] * err_e[:upto]) ** 2).sum(0))

        b = beta[r][:, None]
        total, squares, errors = sums(k[r], r)
        e[r] = b * (v[r] - total)
        err_e[r] = b * np.sqrt((20 * ref.HALF_F32) ** 2 * (squares + v[r] ** 2) + errors)
        total, squares, errors = sums(q[r], r + 1)
        out[r] = total
        err[r] = np.sqrt((13 * ref.HALF_F32) ** 2 * squares + errors)
    return out, err


@pytest.mark.parametrize("max_new", [64, 1], ids=["chunks", "rows"])
@pytest.mark.parametrize("Hk,H,dk,dv", [(2, 4, 128, 128), (4, 4, 64, 96)])
def test_outputs_are_rounded_once(sv, Hk, H, dk, dv, max_new):
    lengths = [64] * 10 + [63, 17, 33, 48, 1]
    c = Rows(lengths, Hk, H, dk, dv, torch.bfloat16, seed=31, far=1e-2)
    c.state *= 5.0  # what the state gives an output, beside what the chunk's rows give
    state = _np(c.state)
    got = _np(sv.gdn_advance(*c.args(), c.state, c.q_start, max_new, state_index=c.index))
    args, start = [_np(t) for t in c.args()], c.q_start.tolist()
    pairs = [_outputs(*(t[r0:r1] for t in args), state[int(slot)])
             for r0, r1, slot in zip(start, start[1:], c.index)]
    want, err = (np.concatenate(t) for t in zip(*pairs))
    assert not (fault := rounding.faults(got[:len(want)], want, err)), fault
    sv.device_status()
