"""kv_pages_step against the sequential reference: whole numbers, so equal."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from gpu_util import dev, sv_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def _state(rng, B, page, max_pages, spare, new, ended=0.0):
    held = rng.integers(0, max_pages + 1, B)
    length = np.array([rng.integers(0, h * page + 1) for h in held])
    n_new = rng.integers(new[0], new[1] + 1, B)
    n_new[rng.random(B) < ended] = -1
    total = int(held.sum()) + spare
    ids = rng.permutation(total)
    table = np.zeros((B, max_pages), np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    ring = np.full(total, -7, np.int32)
    head = int(rng.integers(0, total))
    ring[(head + np.arange(spare)) % total] = ids[at:]
    cursor = np.array([head, spare], np.int32)
    return [a.astype(np.int32) for a in (length, held, cursor, ring, table, n_new)]


def _run(sv, st, page, rows, commit=None, bias=0, in_place=False):
    d = dev()
    length, held, cursor, ring, table, n_new = (torch.from_numpy(a.copy()).to(d) for a in st)
    c = None if commit is None else torch.from_numpy(commit).to(d)
    kw = dict(length_out=length, held_out=held, cursor_out=cursor) if in_place else {}
    r = sv.kv_pages_step(length, held, cursor, ring, table, n_new, page, rows, n_commit=c,
                         n_commit_bias=bias, **kw)
    got = {k: v.cpu().numpy() for k, v in r._asdict().items()}
    got["block_table"], got["ring"] = table.cpu().numpy(), ring.cpu().numpy()
    return got


def _same(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), (k, np.argwhere(got[k] != want[k])[:5].tolist())


@pytest.mark.parametrize("B,page,max_pages,spare,new,rows,ended,seed", [
    (1, 16, 4, 3, (4, 4), 4, 0.0, 0), (1, 16, 1, 1, (1, 1), 7, 0.0, 1),
    (3, 16, 5, 0, (0, 20), 60, 0.3, 2), (32, 64, 9, 40, (4, 4), 130, 0.1, 3),
    (33, 32, 7, 9, (0, 100), 2000, 0.2, 4),     # pages run out
    (64, 16, 6, 500, (1, 90), 1500, 0.0, 5),    # rows run out
    (257, 128, 3, 300, (0, 9), 1400, 0.5, 6), (1000, 16, 20, 3000, (1, 200), 110000, 0.1, 7),
    (4096, 256, 2, 5000, (0, 5), 9000, 0.2, 8), (5, 16, 2000, 9000, (9000, 20000), 90000, 0.0, 9),
])
def test_step_matches(sv, B, page, max_pages, spare, new, rows, ended, seed):
    rng = np.random.default_rng(seed)
    st = _state(rng, B, page, max_pages, spare, new, ended)
    commit = rng.integers(0, 4, B).astype(np.int32)
    for c, bias, place in ((None, 0, False), (commit, 1, True), (commit[:1], -2, False)):
        want = ref.pages_step(*st, page, rows, c, bias)
        _same(_run(sv, st, page, rows, c, bias, place), want)


def test_contradicting_state_is_clamped_and_flagged(sv):
    rng = np.random.default_rng(20)
    st = _state(rng, 6, 16, 3, 4, (1, 5), 0.0)
    st[1][2], st[1][4] = 99, -3          # held out of range
    st[5][5] = -1
    st[4][1, :] = [-5, 1 << 30, 7]       # page ids out of range
    want = ref.pages_step(*st, 16, 30)
    _same(_run(sv, st, 16, 30), want)
    st[2][:] = [-4, 1 << 20]             # the cursor
    want = ref.pages_step(*st, 16, 30)
    assert (want["err_flags"] & 128).all()
    _same(_run(sv, st, 16, 30), want)


def test_steps_in_a_row_captured(sv):
    """A captured step replayed: the state lives in place on the device."""
    d = dev()
    rng = np.random.default_rng(30)
    st = _state(rng, 8, 16, 40, 100, (4, 4))
    t = [torch.from_numpy(a.copy()).to(d) for a in st]
    commit = torch.zeros(8, dtype=torch.int32, device=d)
    bufs = {k: torch.zeros(n, dtype=torch.int32, device=d) for k, n in
            (("q_start", 9), ("kv_len", 8), ("slots", 32), ("positions", 32), ("err_flags", 8))}

    def step():
        sv.kv_pages_step(t[0], t[1], t[2], t[3], t[4], t[5], 16, 32, n_commit=commit,
                         length_out=t[0], held_out=t[1], cursor_out=t[2], **bufs)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    host = [a.copy() for a in st]
    for i in range(6):
        c = rng.integers(0, 5, 8).astype(np.int32)
        commit.copy_(torch.from_numpy(c))
        g.replay()
        w = ref.pages_step(*host, 16, 32, c, 0)
        host[0], host[1], host[2], host[3], host[4] = (w["length"], w["held"], w["cursor"],
                                                       w["ring"], w["block_table"])
        got = {"length": t[0], "held": t[1], "cursor": t[2], "ring": t[3], "block_table": t[4],
               **bufs}
        _same({k: v.cpu().numpy() for k, v in got.items()}, w)
