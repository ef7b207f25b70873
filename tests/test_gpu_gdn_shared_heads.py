"""A layer whose v heads share key heads: a prompt by gdn_advance, then a verify block
through gdn_inputs and the tape, which wants q and k once for each v head."""
import numpy as np
import pytest
import torch

import gdn_ref as ref
from gpu_util import sv_module
from test_gpu_gdn_rows import Layer, _np, _worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def test_verify_block_with_repeated_key_heads(sv):
    Hk, H, dk, dv, W, K = 2, 6, 64, 128, 4, 3
    T, B = K + 1, 2
    prompt = Layer([33, 5], Hk, H, dk, dv, W, torch.float32, seed=70, pad=0)
    prompt.index = torch.arange(B, dtype=torch.int32, device=prompt.x.device)
    prompt.window = prompt.window[:B].contiguous()
    state = torch.zeros(B, H, dv, dk, device=prompt.x.device)
    scale = dk ** -0.5
    sv.gdn_advance(*prompt.run(sv, q_scale=scale, dtype=torch.float32), state, prompt.q_start, 33)
    block = Layer([T] * B, Hk, H, dk, dv, W, torch.float32, seed=71, pad=0)
    r = sv.gdn_inputs(block.x, block.a, block.b, prompt.weight, prompt.window, prompt.a_log, prompt.dt,
                      block.q_start, T, k_heads=Hk, dk=dk, update_window=False, q_scale=scale,
                      dtype=torch.float32)
    before = _np(state)
    q, k = (t.repeat_interleave(H // Hk, 1).unflatten(0, (B, T)) for t in (r.q, r.k))
    out, tape = sv.gdn_tape_capture(state, q, k, *(t.unflatten(0, (B, T)) for t in r[2:]))
    accepted = torch.tensor([0, K], dtype=torch.int32, device=state.device)
    sv.gdn_tape_replay(state, tape, accepted, T, 1)
    # every row's output is that of the packed rows with shared heads
    args = [_np(t) for t in r]
    want, _, out_tol, _ = ref.advance(*args, before, [0, T, 2 * T])
    err = np.abs(_np(out).reshape(want.shape) - want)
    assert _worst(err, out_tol + np.abs(want) * ref.HALF_F32 + 1e-30) <= 1
    # the states, those of the rows that stood
    for b, n in enumerate((1, T)):
        rows = [t[b * T:b * T + n] for t in args]
        _, w_state, _, tol = ref.advance(*rows, before[b:b + 1], [0, n])
        assert _worst(np.linalg.norm(_np(state)[b] - w_state[0], axis=-1), tol[0] + 1e-30) <= 1
    sv.device_status()
