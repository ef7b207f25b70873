"""gdn_inputs, gdn_advance and moe_smallm at the C boundary, on the host: what they
refuse (every call below returns before any launch, on addresses that are never
read), what they do with no rows, and their workspaces' sizes."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    from mtp_speculative_decoding_qmv_gb300 import build as b

    b.build()
    import mtp_speculative_decoding_qmv_gb300 as sv

    assert (sv.SV_F32, sv.SV_BF16) == (F32, BF16)
    return sv.lib()


def at(i):
    """Addresses 4 GiB apart, aligned to 4 KiB."""
    return (i + 1) << 32


# two sequences of ten rows, 2 key heads of 16 and 4 value heads of 8, three slots
INPUTS = dict(x=at(0), a=at(1), b=at(2), x_dtype=BF16, x_stride=96, a_stride=4, b_stride=4,
              weight=at(3), window=at(4), a_log=at(5), dt_bias=at(6), q_start=at(7),
              window_index=at(8), B=2, rows=10, max_new=8, slots=3, W=4, Hk=2, Hv=4, dk=16, dv=8,
              update_window=1, q_scale=1.0, eps=1e-6, out_dtype=BF16, q=at(9), k=at(10), v=at(11),
              alpha=at(12), beta=at(13))


def inputs(L, **kw):
    assert kw.keys() <= INPUTS.keys()
    return L.gdn_inputs(*{**INPUTS, **kw}.values(), None)


@pytest.mark.parametrize("kw", [
    {"B": -1}, {"rows": -1}, {"max_new": -1}, {"slots": -1}, {"Hk": 0}, {"Hv": 0}, {"Hv": 3},
    {"x_dtype": 7}, {"out_dtype": -1}, {"eps": -1.0}, {"eps": float("nan")},
    {"q_scale": float("nan")}, {"window_index": None, "slots": 1},
    {"x": None}, {"a": None}, {"b": None}, {"weight": None}, {"window": None}, {"a_log": None},
    {"dt_bias": None}, {"q_start": None}, {"q": None}, {"k": None}, {"v": None}, {"alpha": None},
    {"beta": None}, {"x_stride": 92}, {"a_stride": 3}, {"b_stride": 3}, {"x_stride": 98},
    {"x_stride": -96}, {"x": at(0) + 8}, {"weight": at(3) + 4}, {"window": at(4) + 8},
    {"q": at(9) + 8}, {"k": at(10) + 2}, {"v": at(11) + 4}, {"a": at(1) + 1}, {"b": at(2) + 1},
    {"a_log": at(5) + 2}, {"dt_bias": at(6) + 1}, {"q_start": at(7) + 2},
    {"window_index": at(8) + 1}, {"alpha": at(12) + 2}, {"beta": at(13) + 2},
    # an output on an input, and on another output: their last bytes too
    {"q": at(0)}, {"k": at(0) + 1904}, {"v": at(3) + 1520}, {"window": at(3)}, {"alpha": at(1)},
    {"beta": at(7)}, {"k": at(9)}, {"v": at(9) + 624}, {"alpha": at(13) + 156}, {"q": at(4) + 3440},
], ids=str)
def test_inputs_refuses(L, kw):
    assert inputs(L, **kw) == INVALID
    assert b"gdn_inputs" in L.sv_last_error()


@pytest.mark.parametrize("kw", [
    {"dk": 4}, {"dv": 0}, {"dk": 12}, {"dv": 136}, {"W": 1}, {"W": 9}, {"Hk": 1, "Hv": 16385}, {"B": 70000, "slots": 70000},
], ids=str)
def test_inputs_does_not_support(L, kw):
    assert inputs(L, **kw) == UNSUPPORTED
    assert b"gdn_inputs" in L.sv_last_error()


ADVANCE = dict(q=at(0), k=at(1), v=at(2), dtype=BF16, q_stride=32, k_stride=32, v_stride=32,
               alpha=at(3), beta=at(4), state=at(5), q_start=at(6), state_index=at(7), B=2,
               rows=100, max_new=80, slots=3, Hk=2, Hv=4, dk=16, dv=8, out=at(8), out_stride=32,
               workspace=at(9), workspace_bytes=1 << 30)


def advance(L, **kw):
    assert kw.keys() <= ADVANCE.keys()
    return L.gdn_advance(*{**ADVANCE, **kw}.values(), None)


@pytest.mark.parametrize("kw", [
    {"B": -1}, {"rows": -1}, {"max_new": -1}, {"slots": -1}, {"Hk": 0}, {"Hv": 0}, {"Hv": 5},
    {"dtype": 9}, {"state_index": None, "slots": 1}, {"q": None}, {"k": None}, {"v": None},
    {"alpha": None}, {"beta": None}, {"state": None}, {"q_start": None}, {"out": None},
    {"q_stride": 24}, {"k_stride": 24}, {"v_stride": 24}, {"out_stride": 24}, {"q_stride": 36},
    {"k_stride": 36}, {"v_stride": 36}, {"out_stride": 36}, {"q": at(0) + 8}, {"k": at(1) + 2},
    {"v": at(2) + 4}, {"state": at(5) + 4}, {"out": at(8) + 8}, {"alpha": at(3) + 2},
    {"beta": at(4) + 1}, {"q_start": at(6) + 1}, {"state_index": at(7) + 2},
    {"workspace": None}, {"workspace": at(9) + 128}, {"workspace_bytes": 0},
    {"workspace_bytes": 100000}, {"workspace": at(5)}, {"workspace": at(8)}, {"workspace": at(0)},
    {"workspace": at(7)}, {"out": at(0)}, {"out": at(2) + 6384}, {"out": at(5)},
    {"out": at(5) + 6128}, {"state": at(1)}, {"state": at(3)}, {"out": at(6)},
], ids=str)
def test_advance_refuses(L, kw):
    assert advance(L, **kw) == INVALID
    assert b"gdn_advance" in L.sv_last_error()


@pytest.mark.parametrize("kw", [
    {"dk": 4}, {"dv": 0}, {"dk": 20}, {"dv": 256}, {"Hk": 1, "Hv": 65536}, {"B": 65535, "slots": 65535},
], ids=str)
def test_advance_does_not_support(L, kw):
    assert advance(L, **kw) == UNSUPPORTED
    assert b"gdn_advance" in L.sv_last_error()


def test_advance_workspace_bytes(L):
    need = L.gdn_advance_workspace_bytes
    assert need(F32, 2, 1000, 1000, 4) == 0 and need(BF16, 200, 200, 1, 4) == 0
    assert need(BF16, -1, 10, 99, 4) == need(BF16, 1, -1, 99, 4) == need(BF16, 1, 10, 99, 0) == 0
    for B, rows, heads in ((1, 1, 1), (1, 64, 3), (1, 65, 3), (5, 5000, 48)):
        # a sequence begins a chunk of its own: at most rows / 64 and one more each
        at_least = 41984 * heads * -(-rows // 64)
        assert at_least <= need(BF16, B, rows, 4000, heads) <= 41984 * heads * (rows // 64 + B + 1)


# ten rows of 256 inputs, 3 of 8 experts of 128
MOE = dict(x=at(0), router=at(1), gate_w=at(2), gate_s=at(3), gate_b=at(4), up_w=at(5), up_s=at(6),
           up_b=at(7), down_w=at(8), down_s=at(9), down_b=at(10), rows=10, hidden=256, inter=128,
           experts=8, top=3, renormalize=1, y=at(11), ids=at(12), weights=at(13),
           workspace=at(14), workspace_bytes=1 << 30)


def moe(L, **kw):
    assert kw.keys() <= MOE.keys()
    return L.moe_smallm(*{**MOE, **kw}.values(), None)


@pytest.mark.parametrize("kw", [
    {"rows": -1}, {"hidden": 0}, {"inter": 0}, {"experts": 0}, {"top": 0}, {"top": 9},
    *[{n: None} for n in list(MOE)[:11]], *[{n: v + 8} for n, v in list(MOE.items())[:11]],
    {"y": None}, {"workspace": None}, {"y": at(11) + 4}, {"ids": at(12) + 2},
    {"weights": at(13) + 1}, {"workspace": at(14) + 64}, {"workspace_bytes": 0},
    {"workspace_bytes": 65536}, {"y": at(0)}, {"y": at(1) + 4088}, {"ids": at(0)},
    {"weights": at(10) + 1020}, {"workspace": at(2)}, {"workspace": at(11)}, {"workspace": at(12)},
    {"ids": at(11) + 5116}, {"weights": at(12) + 116},
], ids=str)
def test_moe_refuses(L, kw):
    assert moe(L, **kw) == INVALID
    assert b"moe_smallm" in L.sv_last_error()


@pytest.mark.parametrize("kw", [
    {"rows": 129}, {"experts": 513}, {"experts": 32, "top": 17}, {"hidden": 192}, {"inter": 64},
    {"hidden": 65536 + 128}, {"inter": 1 << 17},
], ids=str)
def test_moe_does_not_support(L, kw):
    assert moe(L, **kw) == UNSUPPORTED
    assert b"moe_smallm" in L.sv_last_error()


def test_moe_workspace_bytes(L):
    zero = ctypes.c_size_t(7)
    assert L.moe_smallm_workspace_bytes(4, 200, 128, 8, 2, ctypes.byref(zero)) == 0
    assert b"moe_smallm_workspace_bytes" in L.sv_last_error()
    assert L.moe_smallm_workspace_bytes(0, 256, 128, 8, 2, None) > 0
    for sizes in ((1, 128, 128, 1, 1), (128, 2048, 1024, 96, 6), (128, 65536, 128, 512, 16)):
        n = L.moe_smallm_workspace_bytes(*sizes, ctypes.byref(zero))
        # one for more rows serves fewer: no more bytes, and the counters' place is the same
        counters, least = zero.value, L.moe_smallm_workspace_bytes(1, *sizes[1:], ctypes.byref(zero))
        assert least <= n and zero.value == counters
        assert 0 < zero.value < n and zero.value % 256 == n % 256 == 0
        rows, hidden, _, _, top = sizes
        assert n > rows * top * hidden * 4


def test_no_rows_is_a_noop(L):
    none = {n: None for n in ("x", "a", "b", "q", "k", "v", "alpha", "beta")}
    assert inputs(L, rows=0, **none) == OK
    none = {n: None for n in ("q", "k", "v", "out", "alpha", "beta")}
    assert advance(L, rows=0, workspace=None, workspace_bytes=0, **none) == OK
    assert moe(L, rows=0, x=None, y=None, ids=None, weights=None, workspace=None) == OK
