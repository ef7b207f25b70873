"""gdn_inputs, gdn_advance and moe_smallm where calls seldom go: what the Python calls
refuse, rows and states past 32-bit offsets, lengths past the rows, the largest sizes,
graphs that share a workspace, and the three together."""
import numpy as np
import pytest
import torch

import gdn_ref as ref
from gpu_util import dev, sv_module
from test_gpu_gdn_rows import Layer, Rows, _check, _check_inputs, _np
from test_gpu_moe import Layer as Experts
from test_gpu_moe import _check as check_experts

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    return sv_module()


# ---- refusals -----------------------------------------------------------------
def _refused(error, words, call):
    with pytest.raises(error, match=words):
        call()


def test_inputs_refuses(sv):
    c = Layer([3, 4], 2, 4, 16, 8, 4, BF16)
    names = ("x", "a", "b", "weight", "window", "a_log", "dt_bias", "q_start")
    good = dict(zip(names, (c.x, c.a, c.b, c.weight, c.window, c.a_log, c.dt, c.q_start)))
    kept = c.window.clone()

    def call(error, words, change, **kw):
        kw = {"k_heads": 2, "dk": 16, "window_index": c.index, **kw}
        _refused(error, words, lambda: sv.gdn_inputs(*{**good, **change}.values(), 4, **kw))

    call(ValueError, "x must be a CUDA tensor", {"x": c.x.cpu()})
    call(TypeError, "float32 or bfloat16", {"x": c.x.half()})
    call(TypeError, "a must be torch.bfloat16", {"a": c.a.float()})
    call(ValueError, "b has shape", {"b": c.b[:, :3]})
    call(ValueError, "b is on cpu", {"b": c.b.cpu()})
    call(ValueError, "contiguous", {"a": c.a.T.contiguous().T})
    call(TypeError, "weight", {"weight": c.weight.bfloat16()})
    call(ValueError, "window", {"window": c.window[:, :2].contiguous()})
    call(ValueError, "window", {"window": c.window[:, :, ::2]})
    call(ValueError, "a_log", {"a_log": c.a_log[:2]})
    call(TypeError, "dt_bias", {"dt_bias": c.dt.double()})
    call(TypeError, "q_start", {"q_start": c.q_start.long()})
    call(ValueError, "q_start", {"q_start": c.q_start[:0]})
    call(ValueError, "must be", {"x": c.x[0]})
    call(ValueError, "channels", {}, dk=24)
    call(ValueError, "channels", {}, k_heads=0)
    call(ValueError, "needed", {}, dk=None)
    call(TypeError, "window_index", {}, window_index=c.index.long())
    call(ValueError, "window_index", {}, window_index=c.index[:1])
    call(Exception, "W=", {"weight": c.weight[:1], "window": c.window[:, :0]})
    good_out = c.run(sv, update_window=False)
    call(TypeError, "k must be", {}, out=good_out._replace(k=good_out.k.float()))
    call(ValueError, "alpha", {}, out=good_out._replace(alpha=good_out.alpha[:2]))
    call(Exception, "overlap", {}, out=good_out._replace(k=good_out.q))
    assert torch.equal(c.window, kept)


@pytest.mark.parametrize("max_new", [4, 64])
def test_advance_refuses(sv, max_new):
    c = Rows([3, 4], 2, 4, 16, 8, BF16)
    names = ("q", "k", "v", "alpha", "beta", "state", "q_start")
    good = dict(zip(names, (*c.args(), c.state, c.q_start)))
    kept = c.state.clone()

    def call(error, words, change, **kw):
        kw = {"state_index": c.index, **kw}
        _refused(error, words, lambda: sv.gdn_advance(*{**good, **change}.values(), max_new, **kw))

    call(ValueError, "q must be a CUDA tensor", {"q": c.q.cpu()})
    call(TypeError, "float32 or bfloat16", {"q": c.q.half()})
    call(TypeError, "k must be", {"k": c.k.float()})
    call(ValueError, "v has shape", {"v": c.v[:, :3]})
    call(ValueError, "contiguous", {"k": c.k.transpose(1, 2).contiguous().transpose(1, 2)})
    call(TypeError, "alpha", {"alpha": c.alpha.bfloat16()})
    call(ValueError, "beta", {"beta": c.beta[:4]})
    call(ValueError, "state", {"state": c.state[:, :, :, :8]})
    call(TypeError, "state", {"state": c.state.bfloat16()})
    call(ValueError, "must be", {"state": c.state[0]})
    call(TypeError, "q_start", {"q_start": c.q_start.long()})
    call(ValueError, "q_start", {"q_start": c.q_start[:0]})
    call(TypeError, "state_index", {}, state_index=c.index.long())
    call(ValueError, "state_index", {}, state_index=c.index[:1])
    call(TypeError, "out", {}, out=torch.empty_like(c.v, dtype=F32))
    call(ValueError, "out", {}, out=torch.empty_like(c.v)[1:])
    call(Exception, "overlaps", {}, out=c.v)
    if max_new == 64:
        call(Exception, "workspace", {}, workspace=torch.empty(256, dtype=torch.uint8, device=dev()))
        call(TypeError, "workspace", {}, workspace=torch.empty(1 << 20, dtype=F32, device=dev()))
    assert torch.equal(c.state, kept)


def test_experts_refuses(sv):
    c = Experts(3, 256, 128, 8, 2)
    ws = sv.make_moe_workspace(*c.sizes, dev())

    def call(error, words, **kw):
        good = dict(x=c.x, router=c.router, gate=c.gate, up=c.up, down=c.down, top_k=2, workspace=ws)
        good.update(kw)
        _refused(error, words, lambda: sv.moe_smallm(**good))

    call(ValueError, "x must be", x=c.x[0])
    call(ValueError, "x must be a CUDA tensor", x=c.x.cpu())
    call(TypeError, "x must be torch.bfloat16", x=c.x.float())
    call(ValueError, "contiguous", x=c.x.T.contiguous().T)
    call(ValueError, "router", router=c.router[:, :128])
    call(TypeError, "gate w_packed", gate=(c.gate[0].long(), *c.gate[1:]))
    call(TypeError, "up scales", up=(c.up[0], c.up[1].float(), c.up[2]))
    call(ValueError, "down biases", down=(*c.down[:2], c.down[2][:4]))
    call(ValueError, "up w_packed", up=c.down)
    call(TypeError, "ids", ids=torch.empty(3, 2, dtype=torch.int64, device=dev()))
    call(ValueError, "weights", weights=torch.empty(3, 3, device=dev()))
    call(ValueError, "out", out=torch.empty(4, 256, dtype=BF16, device=dev()))
    call(Exception, "top_k", top_k=0)
    call(Exception, "top_k", top_k=9)
    call(Exception, "workspace", workspace=ws[:1024])
    call(TypeError, "workspace", workspace=ws.view(torch.int32))
    call(Exception, "overlap", out=c.x)
    _refused(Exception, "rows", lambda: sv.moe_smallm_workspace_bytes(129, 256, 128, 8, 2))
    n, zero = sv.moe_smallm_workspace_bytes(*c.sizes)
    assert not ws[:zero].any()


# ---- rows -----------------------------------------------------------------------
@pytest.mark.parametrize("dtype,max_new", [(F32, 9), (BF16, 9), (BF16, 100)], ids=str)
def test_lengths_past_the_rows_end_with_them(sv, dtype, max_new):
    """q_start is clamped to [0, rows]."""
    c = Rows([40, 30], 1, 2, 64, 64, dtype, seed=1, pad=0)
    c.q_start = torch.tensor([-5, 40, 1000], dtype=torch.int32, device=dev())
    want = c.want()
    out = sv.gdn_advance(*c.args(), c.state, c.q_start, max_new, state_index=c.index)
    _check(out, c.state, want, dtype)
    i = Layer([40, 30], 1, 2, 64, 64, 4, dtype, seed=2, pad=0)
    i.q_start, i.max_new = c.q_start, max_new
    want = i.want()
    _check_inputs(i.run(sv, dtype=dtype), i.window, want, dtype, 4)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_inputs_without_sequences_are_zeros(sv, dtype):
    c = Layer([5], 2, 2, 16, 16, 4, dtype, seed=3)
    c.q_start, c.index = c.q_start[:1], c.index[:0]
    kept = c.window.clone()
    out = c.run(sv, dtype=dtype)
    assert all((t == 0).all() for t in out) and torch.equal(c.window, kept)


@pytest.mark.parametrize("dtype,max_new", [(F32, 4), (BF16, 4), (BF16, 64)], ids=str)
def test_a_sequence_without_a_slot(sv, dtype, max_new):
    c = Rows([3, 70, 2], 1, 2, 128, 128, dtype, seed=4)
    for bad in (-1, 5, 1 << 30, -(1 << 31)):
        index = c.index.clone()
        index[1] = bad
        before = c.state.clone()
        w_out, w_state, out_tol, tol = ref.advance(*map(_np, c.args()), _np(before), _np(c.q_start), _np(index),
                                                   64 if dtype == BF16 else 1)
        out = sv.gdn_advance(*c.args(), c.state, c.q_start, max_new, state_index=index)
        assert (out[3:73] == 0).all()
        _check(out, c.state, (w_out, w_state, out_tol, tol), dtype)


@pytest.mark.parametrize("n", [1, 100])
def test_states_past_32_bits(sv, n):
    """A slot more than 2^32 bytes into the states."""
    c = Rows([n], 1, 48, 128, 128, BF16, seed=5, pad=0)
    slots = 1500  # 3 MiB each
    state = torch.empty(slots, 48, 128, 128, device=dev())
    state[1498:].fill_(7.0)
    state[1499] = c.state[int(c.index[0])]
    index = torch.tensor([1499], dtype=torch.int32, device=dev())
    out = sv.gdn_advance(*c.args(), state, c.q_start, n, state_index=index)
    want = sv.gdn_advance(*c.args(), c.state, c.q_start, n, state_index=c.index)
    assert torch.equal(out, want) and torch.equal(state[1499], c.state[int(c.index[0])])
    assert (state[1498] == 7.0).all()


@pytest.mark.parametrize("max_new", [1, 2200])
def test_rows_past_32_bits(sv, max_new):
    """Rows 2 MiB apart: the last begin past 2^32 bytes, and (fp32) 4 MiB."""
    c = Rows([2200], 1, 2, 64, 64, BF16, seed=6, pad=1)
    kept = c.state.clone()
    want = sv.gdn_advance(*c.args(), c.state, c.q_start, max_new, state_index=c.index)
    after, c.state = c.state, kept
    far = torch.empty(c.rows, 1 << 20, dtype=BF16, device=dev())
    parts = []
    for i, t in enumerate((c.q, c.k, c.v)):
        view = far[:, 4096 * i:4096 * i + t[0].numel()].unflatten(1, t.shape[1:])
        view.copy_(t)
        parts.append(view)
    out = torch.empty(c.rows, 1 << 20, dtype=BF16, device=dev())
    view = out[:, 8:8 + 128].unflatten(1, (2, 64))
    sv.gdn_advance(*parts, c.alpha, c.beta, c.state, c.q_start, max_new, state_index=c.index, out=view)
    assert torch.equal(view, want) and torch.equal(c.state, after)


def test_inputs_rows_past_32_bits(sv):
    c = Layer([1100], 1, 2, 64, 64, 4, F32, seed=7, pad=1)
    kept = c.window.clone()
    want = c.run(sv)
    after, c.window = c.window, kept
    far = torch.empty(c.rows, 1 << 20, device=dev())
    for i, name in enumerate(("x", "a", "b")):
        t = getattr(c, name)
        view = far[:, 4096 * i:4096 * i + t.shape[1]]
        view.copy_(t)
        setattr(c, name, view)
    got = c.run(sv)
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and torch.equal(c.window, after)


# ---- calls and graphs ------------------------------------------------------------
def test_calls_with_everything_given_allocate_nothing(sv):
    c = Rows([70, 3], 2, 2, 128, 128, BF16, seed=8)
    i = Layer([70, 3], 2, 2, 128, 128, 4, BF16, seed=9)
    e = Experts(5, 256, 128, 8, 2, seed=10)
    outs, out, y = i.run(sv), torch.empty_like(c.v), torch.empty_like(e.x)
    n = sv.gdn_advance_workspace_bytes(BF16, 2, c.rows, c.max_new, 2)
    space, ws = torch.empty(n, dtype=torch.uint8, device=dev()), sv.make_moe_workspace(*e.sizes, dev())
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before = count()
    i.run(sv, out=outs)
    sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index, out=out, workspace=space)
    e.run(sv, out=y, workspace=ws)
    assert count() == before


def test_two_graphs_share_a_workspace(sv):
    """Replayed one after the other, on one stream."""
    long, short = Rows([90, 64], 1, 2, 128, 128, BF16, seed=11), Rows([33, 200], 1, 2, 128, 128, BF16, seed=12)
    n = max(sv.gdn_advance_workspace_bytes(BF16, 2, c.rows, c.max_new, 2) for c in (long, short))
    space = torch.empty(n, dtype=torch.uint8, device=dev())
    a, b = Experts(7, 512, 256, 12, 3, seed=13), Experts(7, 512, 256, 12, 3, seed=14)
    ws = sv.make_moe_workspace(*a.sizes, dev())
    kept = [c.state.clone() for c in (long, short)]
    want = [sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index)
            for c in (long, short)]
    y = [e.run(sv, workspace=ws) for e in (a, b)]
    outs, ys, graphs = [torch.empty_like(t) for t in want], [torch.empty_like(t) for t in y], []
    for i, (c, e) in enumerate(((long, a), (short, b))):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sv.gdn_advance(*c.args(), c.state, c.q_start, c.max_new, state_index=c.index, out=outs[i],
                           workspace=space)
            e.run(sv, out=ys[i], workspace=ws)
    for order in ((0, 1, 1, 0), (1, 0, 0, 1)):
        for i in order:
            (long, short)[i].state.copy_(kept[i])
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(outs + ys, want + y))
    sv.device_status()


# ---- experts ---------------------------------------------------------------------
@pytest.mark.parametrize("rows,hidden,inter,experts,top", [
    (2, 65536, 128, 3, 2), (1, 128, 65536, 2, 1), (128, 128, 128, 512, 16), (16, 256, 128, 16, 16)])
def test_experts_largest_sizes(sv, rows, hidden, inter, experts, top):
    c = Experts(rows, hidden, inter, experts, top, seed=15)
    check_experts(c, c.run(sv))
    sv.device_status()


def test_a_workspace_of_more_rows_serves_fewer(sv):
    layers = [Experts(rows, 512, 384, 20, 3, seed=rows) for rows in (128, 3, 100, 1, 17, 128)]
    ws = sv.make_moe_workspace(128, 512, 384, 20, 3, dev())
    for e in layers:
        check_experts(e, e.run(sv, workspace=ws))
    n, zero = sv.moe_smallm_workspace_bytes(128, 512, 384, 20, 3)
    assert not ws[:zero].any()
    sv.device_status()


@pytest.mark.parametrize("rows", [1, 7, 40])
def test_experts_of_zero_inputs_and_wide_ranges(sv, rows):
    """Groups of zeros, and groups whose values span 2^24."""
    c = Experts(rows, 512, 256, 6, 2, seed=16)
    c.x[:, 64:128] = 0.0
    c.x[:, 128:192] *= (2.0 ** -torch.arange(0, 64, device=dev()).clamp(max=24)).bfloat16()
    check_experts(c, c.run(sv))
    c.x.zero_()
    assert (c.run(sv) == 0).all()


# ---- together --------------------------------------------------------------------
def test_a_block_of_both_in_a_graph(sv):
    """A step of mixed rows through a GatedDeltaNet layer and the experts after it,
    captured; every operator against its reference on what it was given."""
    H, d, lengths = 2, 128, [1, 40, 4, 0, 1]
    c = Layer(lengths, 1, H, d, d, 4, BF16, seed=17, pad=3)
    e = Experts(c.rows, H * d, 128, 10, 3, seed=18)
    state = torch.randn(len(lengths) + 2, H, d, d, device=dev()) * 0.1
    ws, window0, state0 = sv.make_moe_workspace(*e.sizes, dev()), c.window.clone(), state.clone()

    def step():
        w = c.run(sv, q_scale=d ** -0.5)
        o = sv.gdn_advance(*w, state, c.q_start, c.max_new, state_index=c.index)
        e.x = o.flatten(1)
        return w, o, e.run(sv, workspace=ws)

    eager = step()
    window1, state1 = c.window.clone(), state.clone()
    c.window.copy_(window0)
    want = c.want(q_scale=d ** -0.5)
    _check_inputs(eager[0], window1, want, BF16, 4)
    want = ref.advance(*map(_np, eager[0]), _np(state0), _np(c.q_start), _np(c.index), 64)
    _check(eager[1], state1, want, BF16)
    check_experts(e, eager[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        c.window.copy_(window0)
        state.copy_(state0)
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip((*captured[0], *captured[1:]), (*eager[0], *eager[1:])):
            assert torch.equal(g, w)
        assert torch.equal(state, state1) and torch.equal(c.window, window1)
    assert np.all(_np(eager[1][-3:]) == 0)
    sv.device_status()
