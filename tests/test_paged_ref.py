"""The paged-cache operators on the host: the references pinned by hand-worked
cases, the frequency words, and the C ABI's refusals (no GPU: every call below
returns during host-side validation)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_ref as ref


def _i32(*v):
    return np.array(v, np.int32)


def test_pages_step_worked_example():
    # page 16; request 0 holds one page with 14 tokens, commits 1 (+1): 16; 4 new
    # tokens need a second page; request 1 ended with 2 pages; request 2 is new
    table = np.array([[5, 0, 0], [1, 2, 0], [0, 0, 0]], np.int32)
    ring = _i32(7, 6, 3, 0, 0, 0, 0, 4)  # head 7: free pages 4, 7, 6
    r = ref.pages_step(_i32(14, 20, 0), _i32(1, 2, 0), _i32(7, 3), ring, table, _i32(4, -1, 17),
                       16, 23, _i32(1, 0, -1), 1)
    assert r["length"].tolist() == [16, 0, 0] and r["held"].tolist() == [2, 0, 2]
    assert r["kv_len"].tolist() == [20, 0, 17] and r["q_start"].tolist() == [0, 4, 4, 21]
    assert r["block_table"][0, :2].tolist() == [5, 4] and r["block_table"][2, :2].tolist() == [7, 6]
    assert r["slots"].tolist() == [64, 65, 66, 67, *range(112, 128), 96, -1, -1]
    assert r["positions"].tolist() == [16, 17, 18, 19, *range(17), 0, 0]
    assert r["cursor"].tolist() == [2, 2] and r["ring"][2:4].tolist() == [1, 2]
    assert r["err_flags"].tolist() == [0, 0, 0]


def test_pages_step_refusals():
    table = np.zeros((4, 2), np.int32)
    r = ref.pages_step(_i32(0, 0, 0, 0), _i32(0, 0, 0, 0), _i32(0, 2), _i32(0, 1, 2, 3), table,
                       _i32(16, 33, 30, 3), 16, 82)
    # request 1 passes max_pages; 2 wants two pages of the one left; 3 comes after it
    assert r["err_flags"].tolist() == [0, 32, 32, 32] and r["kv_len"].tolist() == [16, 0, 0, 0]
    assert r["q_start"].tolist() == [0, 16, 49, 79, 82] and r["cursor"].tolist() == [1, 1]
    r = ref.pages_step(_i32(0, 0), _i32(0, 0), _i32(0, 4), _i32(0, 1, 2, 3), table[:2], _i32(3, 9),
                       16, 10)
    assert r["err_flags"].tolist() == [0, 64] and r["q_start"].tolist() == [0, 3, 10]
    assert r["slots"].tolist() == [0, 1, 2] + [-1] * 7


def test_rotate_quarter_turns():
    x = np.arange(1.0, 17.0).reshape(1, 1, 16)
    out, _ = ref.rotate(x, np.array([1]), np.array([math.pi / 2]), interleaved=False)
    assert np.allclose(out[0, 0, :2], [-2, 1]) and np.array_equal(out[0, 0, 2:], x[0, 0, 2:])
    out, _ = ref.rotate(x, np.array([[3, 1]]), np.array([math.pi / 2, math.pi]), axis=[1, 0],
                        interleaved=True)
    assert np.allclose(out[0, 0, :4], [-2, 1, -3, -4])


def test_attention_of_equal_keys_is_the_mean():
    k = np.ones((3, 1, 16, 64))
    v = np.random.default_rng(0).normal(size=(3, 1, 16, 64))
    table = np.array([[2, 0, -1]], np.int32)
    q = np.ones((2, 1, 64))
    out, lse, _, _ = ref.attention(q, k, v, table, [0, 2], [20], 0.25)
    both = np.concatenate([v[2, 0], v[0, 0]])
    assert np.allclose(out[0, 0], both[:19].mean(0)) and np.allclose(out[1, 0], both[:20].mean(0))
    assert np.allclose(lse[:, 0], [16 + math.log(19), 16 + math.log(20)])
    out, lse, _, _ = ref.attention(q, k, v, table, [0, 2], [1], 0.25, window=5)
    assert (out[0] == 0).all() and np.isneginf(lse[0, 0]) and np.allclose(out[1, 0], v[2, 0, 0])


def test_rope_freqs_are_exact_turns():
    import mtp_speculative_decoding_qmv_gb300 as sv

    inv = torch.tensor([1.0, 0.1234567, 1e-6, 3.9, 0.0, 2 * math.pi], dtype=torch.float64)
    words = sv.rope_freqs(inv)
    assert words.dtype == torch.int64
    two_pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50) * 2
    for f, w in zip(inv.tolist(), words.tolist()):
        turns = Fraction(f) / two_pi
        off = (Fraction(w % 2 ** 64, 2 ** 64) - turns) % 1
        off = min(off, 1 - off)
        assert off <= Fraction(2) ** -52, f  # the quotient's double rounding
    with pytest.raises(TypeError):
        sv.rope_freqs(inv.float())


# ---- refusals ---------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    from mtp_speculative_decoding_qmv_gb300 import build as b

    b.build()
    import mtp_speculative_decoding_qmv_gb300 as sv

    return sv.lib()


A = 1 << 32  # fake device addresses, never dereferenced here
M = 1 << 28


def _pages(L, length=A, held=A + M, cursor=A + 2 * M, n_new=A + 3 * M, commit=A + 4 * M,
           n_commit=8, B=8, page=16, max_pages=10, num_pages=100, rows=40, table=A + 5 * M,
           ring=A + 6 * M, length_out=A, held_out=A + M, cursor_out=A + 2 * M, q_start=A + 7 * M,
           kv_len=A + 8 * M, slots=A + 9 * M, positions=A + 10 * M, flags=A + 11 * M):
    return L.kv_pages_step(length, held, cursor, n_new, commit, n_commit, 1, B, page, max_pages,
                           num_pages, rows, table, ring, length_out, held_out, cursor_out,
                           q_start, kv_len, slots, positions, flags, None)


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"rows": -1}, 1), ({"max_pages": 0}, 1), ({"num_pages": 0}, 1),
    ({"page": 24}, 2), ({"page": 8}, 2), ({"page": 512}, 2), ({"B": 4097}, 2),
    ({"max_pages": 1 << 27}, 2), ({"num_pages": 1 << 27}, 2), ({"n_commit": 0}, 1),
    ({"n_commit": 9}, 1), ({"length": 0}, 1), ({"ring": 0}, 1), ({"slots": 0}, 1),
    ({"positions": A + 10 * M + 2}, 1), ({"n_new": A + 3 * M + 1}, 1),
    ({"slots": A + 10 * M}, 1), ({"length_out": A + 4}, 1), ({"held_out": A}, 1),
    ({"kv_len": A + 3 * M}, 1), ({"flags": A + 8 * M + 8}, 1), ({"table": A + 6 * M + 4}, 1),
])
def test_kv_pages_step_rejects(L, kw, status):
    assert _pages(L, **kw) == status
    assert L.sv_last_error() != b""


def test_kv_pages_step_empty(L):
    assert _pages(L, B=0) == 0


def _rope(L, q=A, k=A + M, v=A + 2 * M, dt=1, qs=1024, ks=256, vs=256, pos=A + 3 * M, axes=1,
          slots=A + 4 * M, freqs=A + 5 * M, axis=0, qw=0, kw=0, eps=1e-6, rows=4, Hq=8, Hkv=2,
          D=128, R=128, inter=0, page=16, pages=10, qo=A + 6 * M, kc=A + 7 * M, vc=A + 8 * M):
    return L.rope_kv_append(q, k, v, dt, qs, ks, vs, pos, axes, slots, freqs, axis, qw, kw, eps,
                            rows, Hq, Hkv, D, R, inter, page, pages, qo, kc, vc, None)


@pytest.mark.parametrize("kw,status", [
    ({"rows": -1}, 1), ({"Hq": 0}, 1), ({"Hkv": 0}, 1), ({"pages": 0}, 1), ({"dt": 5}, 1),
    ({"D": 96}, 2), ({"R": 24}, 1), ({"R": 144}, 1), ({"R": -16}, 1), ({"axes": 0}, 2),
    ({"axes": 5}, 2), ({"page": 48}, 2), ({"pages": 1 << 27}, 2), ({"Hq": 5000, "qs": 640000}, 2),
    ({"eps": -1.0}, 1), ({"eps": float("nan")}, 1), ({"q": 0}, 1), ({"freqs": 0}, 1),
    ({"axes": 3, "axis": 0}, 1), ({"qs": 1000}, 1), ({"ks": 260}, 1), ({"q": A + 8}, 1),
    ({"kc": A + 7 * M + 2}, 1), ({"pos": A + 3 * M + 1}, 1), ({"freqs": A + 5 * M + 4}, 1),
    ({"qo": A}, 1), ({"vc": A + 7 * M}, 1), ({"kc": A + 2 * M}, 1),
])
def test_rope_kv_append_rejects(L, kw, status):
    assert _rope(L, **kw) == status
    assert L.sv_last_error() != b""


def test_rope_kv_append_empty(L):
    assert _rope(L, rows=0) == 0


def _attend(L, q=A, qs=1024, kc=A + M, vc=A + 2 * M, table=A + 3 * M, q_start=A + 4 * M,
            kv_len=A + 5 * M, B=2, rows=8, max_new=4, Hq=8, Hkv=2, D=128, page=16, pages=100,
            max_pages=10, scale=0.1, window=0, out=A + 6 * M, os=1024, lse=A + 7 * M,
            ws=A + 8 * M, nbytes=1 << 30):
    return L.paged_attention(q, qs, kc, vc, table, q_start, kv_len, B, rows, max_new, Hq, Hkv, D,
                             page, pages, max_pages, scale, window, out, os, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"rows": -1}, 1), ({"max_new": -1}, 1), ({"Hq": 0}, 1), ({"Hkv": 3}, 1),
    ({"pages": 0}, 1), ({"max_pages": 0}, 1), ({"D": 80}, 2), ({"page": 20}, 2),
    ({"scale": 0.0}, 1), ({"scale": -1.0}, 1), ({"scale": float("inf")}, 1),
    ({"scale": float("nan")}, 1), ({"window": -1}, 1), ({"pages": 1 << 26}, 2),
    ({"max_pages": 1 << 27}, 2), ({"rows": 1 << 30}, 2), ({"max_pages": (1 << 27) - 17, "rows": 16}, 2),
    ({"scale": 2.5e38}, 1), ({"q": 0}, 1), ({"ws": 0}, 1),
    ({"qs": 1016}, 1), ({"os": 1028}, 1), ({"kc": A + M + 8}, 1), ({"out": A + 6 * M + 4}, 1),
    ({"lse": A + 7 * M + 2}, 1), ({"ws": A + 8 * M + 128}, 1), ({"nbytes": 4096}, 1),
    ({"out": A}, 1), ({"lse": A + 4 * M}, 1), ({"ws": A + M}, 1), ({"lse": A + 6 * M}, 1),
])
def test_paged_attention_rejects(L, kw, status):
    assert _attend(L, **kw) == status
    assert L.sv_last_error() != b""


def test_paged_attention_empty(L):
    assert _attend(L, B=0) == 0 and _attend(L, rows=0) == 0


def test_paged_attention_workspace_bytes(L):
    assert L.paged_attention_workspace_bytes(96) == 0
    sizes = [L.paged_attention_workspace_bytes(D) for D in (64, 128, 256)]
    assert all(n > 4096 for n in sizes)


def test_binding_refuses_host_tensors():
    import mtp_speculative_decoding_qmv_gb300 as sv

    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.kv_pages_step(z, z, torch.zeros(2, dtype=torch.int32), z, z[None], z, 16, 1)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.rope_kv_append(x, x, x, z, z, None, c, c)
    with pytest.raises(ValueError):
        sv.paged_attention(x, c, c, z[None], torch.zeros(2, dtype=torch.int32), z, 1)
