"""gdn_inputs and gdn_advance over packed rows against float64."""
import numpy as np
import pytest
import torch

import gdn_ref as ref
from gpu_util import dev, sv_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def _np(t):
    return t.detach().double().cpu().numpy()


def _worst(err, bound):
    return float(np.where(np.isnan(err), np.inf, err / bound).max())


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=dev(), dtype=dtype)


class Rows:
    """Sequences of the given lengths, slots in any order among two more, and
    `pad` rows past the last."""

    def __init__(self, lengths, Hk, H, dk, dv, dtype, seed=0, pad=2, far=1e-3):
        d, g = dev(), torch.Generator(device=dev())
        g.manual_seed(seed)
        starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        self.lengths, self.rows, self.max_new = lengths, int(starts[-1]) + pad, max(lengths)
        self.q_start = torch.from_numpy(starts).to(d)
        self.index = torch.randperm(len(lengths) + 2, generator=g, device=d)[:len(lengths)].int()
        unit = lambda h: torch.nn.functional.normalize(_randn(g, self.rows, h, dk), dim=-1)  # noqa: E731
        self.q, self.k = (unit(Hk) / dk ** 0.5).to(dtype), unit(Hk).to(dtype)
        self.v = _randn(g, self.rows, H, dv, dtype=dtype)
        rate = far ** torch.rand(H, generator=g, device=d)
        self.alpha = torch.exp(-rate * torch.nn.functional.softplus(_randn(g, self.rows, H)))
        self.beta = torch.sigmoid(_randn(g, self.rows, H))
        self.state = _randn(g, len(lengths) + 2, H, dv, dk) * 0.1

    def args(self):
        return self.q, self.k, self.v, self.alpha, self.beta

    def want(self):
        return ref.advance(*map(_np, self.args()), _np(self.state), _np(self.q_start),
                           _np(self.index), 64 if self.q.dtype == torch.bfloat16 else 1)


def _check(out, state, want, dtype):
    w_out, w_state, out_tol, tol = want
    rounding = ref.HALF_BF16 if dtype == torch.bfloat16 else ref.HALF_F32
    bound = out_tol + np.abs(w_out) * rounding + 1e-30
    assert _worst(np.abs(_np(out) - w_out), bound) <= 1
    assert _worst(np.linalg.norm(_np(state) - w_state, axis=-1), tol + 1e-30) <= 1


LENGTHS = [[1], [1, 1, 1], [0, 3, 0, 1], [16, 5], [31], [32], [63, 64, 65], [1, 0, 200, 40], [129],
           [333, 2, 64, 1]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_advance_lengths(sv, lengths, dtype):
    c = Rows(lengths, 2, 4, 128, 128, dtype, seed=sum(lengths))
    want = c.want()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
    _check(out, c.state, want, dtype)
    assert (out[-2:] == 0).all()
    sv.device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Hk,H,dk,dv", [(1, 1, 8, 8), (1, 3, 64, 64), (3, 3, 64, 128), (2, 2, 128, 64),
                                        (1, 2, 96, 80), (2, 4, 120, 104), (5, 5, 16, 128)])
def test_advance_heads(sv, Hk, H, dk, dv, dtype):
    for lengths in ([3, 1], [70, 0, 150]):
        c = Rows(lengths, Hk, H, dk, dv, dtype, seed=dk + dv)
        want = c.want()
        out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
        _check(out, c.state, want, dtype)
    sv.device_status()


def test_advance_a_prompt_in_pieces_is_the_prompt(sv):
    """Chunks of a prompt, then single tokens, against the whole."""
    c = Rows([400], 2, 2, 128, 128, torch.bfloat16, seed=5, pad=0)
    state, tol, at = _np(c.state), 0.0, 0
    for n in (130, 64, 1, 7, 150, 1, 47):
        part = [t[at:at + n] for t in c.args()]
        start = torch.tensor([0, n], dtype=torch.int32, device=dev())
        out = sv.gdn_advance(*part, c.state, start, n, state_index=c.index)
        want = ref.advance(*map(_np, part), state, [0, n], _np(c.index), 64, tol)
        _check(out, c.state, want, torch.bfloat16)
        state, tol, at = want[1], want[3], at + n


def test_advance_long(sv):
    c = Rows([3000, 1000], 1, 2, 128, 128, torch.bfloat16, seed=6)
    want = c.want()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
    _check(out, c.state, want, torch.bfloat16)


@pytest.mark.parametrize("lengths", [[5, 9], [70, 130]], ids=str)
@pytest.mark.parametrize("gate", [0.0, 1.0, 1e-30])
def test_advance_gates_at_their_ends(sv, lengths, gate):
    """alpha 0 forgets everything, alpha 1 nothing; beta 0 and 1."""
    c = Rows(lengths, 2, 2, 128, 128, torch.bfloat16, seed=7)
    c.alpha[::3] = gate
    c.beta[1::4] = 0.0
    c.beta[2::5] = 1.0
    want = c.want()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
    _check(out, c.state, want, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[5, 3], [70, 100]], ids=str)
def test_advance_strided_rows_and_what_lies_between(sv, lengths, dtype):
    """q, k, v as slices of one row, out as a slice: the gaps hold NaN and stay."""
    H, dk, dv = 2, 64, 128
    c = Rows(lengths, H, H, dk, dv, dtype, seed=8)
    want = c.want()
    wide = torch.full((c.rows, 2 * H * dk + H * dv + 16), float("nan"), dtype=dtype, device=dev())
    q = wide[:, :H * dk].unflatten(1, (H, dk))
    k = wide[:, H * dk:2 * H * dk].unflatten(1, (H, dk))
    v = wide[:, 2 * H * dk:2 * H * dk + H * dv].unflatten(1, (H, dv))
    for to, t in ((q, c.q), (k, c.k), (v, c.v)):
        to.copy_(t)
    # the padding rows hold what they may
    for t in (q, k, v, c.alpha, c.beta):
        t[-2:] = float("nan")
    to = torch.full((c.rows, H * dv + 8), 7.0, dtype=dtype, device=dev())
    out = sv.gdn_advance(q, k, v, c.alpha, c.beta, c.state, c.q_start, c.max_new,
                         state_index=c.index, out=to[:, :H * dv].unflatten(1, (H, dv)))
    _check(out, c.state, want, dtype)
    assert (to[:, H * dv:] == 7).all() and (out[-2:] == 0).all()


@pytest.mark.parametrize("lengths", [[3, 4, 2], [70, 80, 64]], ids=str)
def test_advance_sequences_do_not_meet(sv, lengths):
    """A sequence without a slot, and one full of NaN, beside others."""
    c = Rows(lengths, 2, 2, 128, 128, torch.bfloat16, seed=9)
    want = c.want()
    r0, r1, r2 = np.cumsum([0] + lengths)[:3]
    kept = c.state.clone()
    bad = int(c.index[0])
    c.index[0] = 99
    for t in c.args():
        t[r1:r2] = float("nan")
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
    assert (out[r0:r1] == 0).all() and torch.equal(c.state[bad], kept[bad])
    assert out[r1:r2].isnan().all() and c.state[int(c.index[1])].isnan().all()
    third = int(c.index[2])
    bound = want[2][r2:-2] + np.abs(want[0][r2:-2]) * ref.HALF_BF16
    assert _worst(np.abs(_np(out[r2:-2]) - want[0][r2:-2]), bound) <= 1
    off = np.linalg.norm(_np(c.state[third]) - want[1][third], axis=-1)
    assert _worst(off, want[3][third]) <= 1
    unused = [s for s in range(5) if s not in c.index.tolist()]
    assert torch.equal(c.state[unused], kept[unused])


def test_advance_without_index_or_sequences(sv):
    c = Rows([4, 70], 1, 1, 128, 128, torch.bfloat16, seed=10)
    c.index = torch.arange(2, dtype=torch.int32, device=dev())
    want = c.want()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new)
    _check(out, c.state, want, torch.bfloat16)
    kept = c.state.clone()
    for n in (1, 64):
        out = sv.gdn_advance(*c.args(), c.state, c.q_start[:1], n)
        assert (out == 0).all() and torch.equal(c.state, kept)
    none = sv.gdn_advance(*(t[:0] for t in c.args()), c.state, c.q_start[:1], 0)
    assert none.shape == (0, 1, 128)


@pytest.mark.parametrize("max_new", [0, 1, 1000])
def test_advance_max_new_only_picks_the_kernel(sv, max_new):
    c = Rows([1, 90, 0, 33], 1, 2, 128, 128, torch.bfloat16, seed=11)
    want = c.want()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, max_new, state_index=c.index)
    _check(out, c.state, want, torch.bfloat16)


@pytest.mark.parametrize("lengths", [[2, 1, 3], [500, 70, 1]], ids=str)
def test_advance_repeats_to_the_bit_in_a_graph_and_on_streams(sv, lengths):
    c = Rows(lengths, 2, 4, 128, 128, torch.bfloat16, seed=12)
    kept = c.state.clone()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
    want, after = out.clone(), c.state.clone()
    side = [torch.cuda.Stream() for _ in range(2)]
    states, outs = [kept.clone() for _ in side], [torch.empty_like(out) for _ in side]
    torch.cuda.synchronize()
    for s, st, o in zip(side, states, outs):  # two at once
        with torch.cuda.stream(s):
            for _ in range(5):
                st.copy_(kept)
                sv.gdn_advance(*c.args(), st, c.q_start, c.max_new, state_index=c.index, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(s, after) for s in states)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index, out=out)
    for _ in range(3):
        c.state.copy_(kept)
        out.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.state, after)
    sv.device_status()


# ---- gdn_inputs ---------------------------------------------------------------
class Layer:
    def __init__(self, lengths, Hk, H, dk, dv, W, dtype, seed=0, pad=2):
        d, g = dev(), torch.Generator(device=dev())
        g.manual_seed(seed)
        starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        self.rows, self.max_new, self.Hk, self.dk = int(starts[-1]) + pad, max(lengths), Hk, dk
        self.q_start = torch.from_numpy(starts).to(d)
        self.index = torch.randperm(len(lengths) + 2, generator=g, device=d)[:len(lengths)].int()
        C = 2 * Hk * dk + H * dv
        both = _randn(g, self.rows, C + 2 * H + 2 * H % 4 + 4, dtype=dtype)  # one projection's rows
        self.x, self.a, self.b = both[:, :C], both[:, C:C + H], both[:, C + H:C + 2 * H]
        self.weight = _randn(g, W, C) / W ** 0.5
        self.window = _randn(g, len(lengths) + 2, W - 1, C)
        self.a_log, self.dt = _randn(g, H), _randn(g, H)

    def want(self, **kw):
        return ref.inputs(*map(_np, (self.x, self.a, self.b, self.weight, self.window, self.a_log,
                                     self.dt, self.q_start)), self.Hk, self.dk, _np(self.index), **kw)

    def run(self, sv, **kw):
        return sv.gdn_inputs(self.x, self.a, self.b, self.weight, self.window, self.a_log, self.dt,
                             self.q_start, self.max_new, k_heads=self.Hk, dk=self.dk,
                             window_index=self.index, **kw)


def _check_inputs(got, window, want, dtype, W):
    outs, mags = want
    rounding = ref.HALF_BF16 if dtype == torch.bfloat16 else ref.HALF_F32
    # W products and sums; silu: an exponential and a division of 2 ulp each, the
    # exponent's rounding of up to |y| steps; a norm over 128 terms and its root
    u = (W + 2 * 2 + 16 + 8) * 2 * ref.HALF_F32
    for g, w, m in zip(got[:3], outs[:3], mags):
        bound = np.abs(w) * (rounding + u) + u * m + 1e-30
        assert _worst(np.abs(_np(g) - w), bound) <= 1
    for g, w in zip(got[3:], outs[3:5]):
        # exp of exp times a logarithm: a few steps of the exponent, which is at most 100 here
        bound = 16 * ref.HALF_F32 * (1 + np.abs(np.log(np.maximum(w, 1e-38)))) * w + 1e-37
        assert _worst(np.abs(_np(g) - w), bound) <= 1
    assert np.array_equal(_np(window), outs[5])


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16], ids=["from f32", "from bf16"])
@pytest.mark.parametrize("dst", [torch.float32, torch.bfloat16], ids=["to f32", "to bf16"])
@pytest.mark.parametrize("lengths", [[1], [4], [0, 1, 2, 3, 0, 4], [17, 1, 100, 33], [64, 16, 32]], ids=str)
def test_inputs_lengths(sv, lengths, src, dst):
    c = Layer(lengths, 2, 6, 128, 128, 4, src, seed=sum(lengths))
    want = c.want(q_scale=0.25)
    got = c.run(sv, q_scale=0.25, dtype=dst)
    _check_inputs(got, c.window, want, dst, 4)
    assert all((t[-2:] == 0).all() for t in got)


@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("Hk,H,dk,dv", [(1, 1, 8, 8), (1, 2, 64, 96), (3, 3, 128, 64), (2, 34, 16, 24)])
def test_inputs_shapes(sv, Hk, H, dk, dv, W):
    for lengths in ([1, 5], [40, 0, 3]):
        c = Layer(lengths, Hk, H, dk, dv, W, torch.bfloat16, seed=W)
        want = c.want()
        _check_inputs(c.run(sv, dtype=torch.float32), c.window, want, torch.float32, W)


def test_inputs_window_only_when_asked_and_slots(sv):
    c = Layer([3, 20, 2], 2, 2, 64, 64, 4, torch.float32, seed=3)
    kept = c.window.clone()
    want = c.want(update=False)
    got = c.run(sv, update_window=False, dtype=torch.float32)
    _check_inputs(got, c.window, want, torch.float32, 4)
    assert torch.equal(c.window, kept)
    c.index[1] = -1
    want = c.want()
    _check_inputs(c.run(sv, dtype=torch.float32), c.window, want, torch.float32, 4)


def test_inputs_extreme_gates_and_values(sv):
    c = Layer([5], 1, 4, 64, 64, 4, torch.float32, seed=4, pad=0)
    c.a[:] = torch.tensor([100.0, -100.0, float("inf"), -float("inf")], device=dev())
    c.b[:] = torch.tensor([200.0, -200.0, float("inf"), -float("inf")], device=dev())
    c.a_log[:] = 0.0
    c.x[:, :64] = 0.0          # a head of zeros: eps keeps it zero
    c.window[:, :, :64] = 0.0
    c.x[:, 64:128] *= -1e6     # silu's far side
    got = c.run(sv, dtype=torch.float32)
    assert (got.q == 0).all() and all(t.isfinite().all() for t in got)
    z = torch.tensor([100.0, -100.0, float("inf"), -float("inf")], device=dev()) + c.dt
    want = torch.exp(-torch.nn.functional.softplus(z.double())).float()
    assert torch.allclose(got.alpha[0], want, rtol=1e-4, atol=1e-37)
    assert got.beta[0].tolist() == [1.0, 0.0, 1.0, 0.0]


def test_inputs_many_sequences(sv):
    lengths = [(7 * i) % 5 for i in range(3000)] + [1]
    c = Layer(lengths, 1, 1, 8, 8, 4, torch.bfloat16, seed=5)
    want = c.want()
    _check_inputs(c.run(sv), c.window, want, torch.bfloat16, 4)


# ---- a layer's prompt, then verify cycles --------------------------------------
def test_a_layer_from_its_prompt_through_verify_blocks(sv):
    """A prompt by gdn_inputs and gdn_advance, then verify blocks by the tape,
    some drafts rejected: the states and windows of one run over what stood."""
    H, d, W, lengths, K = 2, 128, 4, [100, 37], 3
    c = Layer(lengths, H, H, d, d, W, torch.float32, seed=21, pad=0)
    c.index = torch.arange(2, dtype=torch.int32, device=dev())
    c.window = c.window[:2].contiguous()
    state = torch.zeros(2, H, d, d, device=dev())
    win0 = c.window.clone()
    w = c.run(sv, q_scale=d ** -0.5)
    sv.gdn_advance(*w, state, c.q_start, max(lengths))
    stood = [[c.x[s:e]] for s, e in zip(c.q_start.tolist(), c.q_start.tolist()[1:])]
    gates = [[c.a[s:e]] for s, e in zip(c.q_start.tolist(), c.q_start.tolist()[1:])]
    bgates = [[c.b[s:e]] for s, e in zip(c.q_start.tolist(), c.q_start.tolist()[1:])]
    T = K + 1
    blocks = torch.arange(0, 2 * T + 1, T, dtype=torch.int32, device=dev())
    for step in range(3):
        v = Layer([T, T], H, H, d, d, W, torch.float32, seed=30 + step, pad=0)
        x = v.x.contiguous()
        r = sv.gdn_inputs(x, v.a, v.b, c.weight, c.window, c.a_log, c.dt, blocks, T, k_heads=H, dk=d,
                          update_window=False, q_scale=d ** -0.5, dtype=torch.float32)
        _, tape = sv.gdn_tape_capture(state, *(t.unflatten(0, (2, T)) for t in r))
        accepted = torch.tensor([step, K - step], dtype=torch.int32, device=dev())
        sv.gdn_tape_replay(state, tape, accepted, T, 1)
        sv.conv_window_replay(c.window, x.unflatten(0, (2, T)), accepted, 1)
        for s in range(2):
            n = int(accepted[s]) + 1
            stood[s].append(x[s * T:s * T + n])
            gates[s].append(v.a[s * T:s * T + n])
            bgates[s].append(v.b[s * T:s * T + n])
    n = [sum(len(t) for t in stood[s]) for s in range(2)]
    flat = lambda lists: torch.cat([t for one in lists for t in one])  # noqa: E731
    (q, k, v, al, be, window), _ = ref.inputs(
        *map(_np, (flat(stood), flat(gates), flat(bgates), c.weight, win0, c.a_log, c.dt)),
        [0, n[0], sum(n)], H, d, q_scale=d ** -0.5)
    _, want, _, _ = ref.advance(q, k, v, al, be, np.zeros((2, H, d, d)), [0, n[0], sum(n)])
    assert np.array_equal(_np(c.window), window)
    # the prompt's k and v are rounded to bf16: half a step of each, in norm
    err = np.linalg.norm(_np(state) - want) / np.linalg.norm(want)
    assert err < 3 * ref.HALF_BF16
    sv.device_status()
