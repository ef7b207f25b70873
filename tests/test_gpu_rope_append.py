"""rope_kv_append against float64: norm, rotary positions, slots.

Bound per element: a bf16 rounding of the result, and 2^-18 of its two terms'
magnitude (angle 2^-25 of a half turn and sincospi's 2 units: 2^-21; three fp32
products and sums 3 x 2^-24; the norm's D / 32 + 9 operations 17 x 2^-24; twice
that for margin)."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from gpu_util import dev, sv_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def _close(got, want, mag):
    tol = ref.HALF_BF16 * np.abs(want) + (1 + ref.HALF_BF16) * 2.0 ** -18 * mag
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:3].tolist())


@pytest.mark.parametrize("rows,Hq,Hkv,D,R,axes,norm,inter,dt,page", [
    (1, 1, 1, 64, 64, 1, False, False, "f32", 16), (4, 40, 40, 128, 128, 1, False, False, "f32", 16),
    (7, 5, 1, 128, 32, 1, True, True, "f32", 32), (33, 8, 2, 64, 16, 3, True, False, "bf16", 64),
    (130, 20, 4, 256, 64, 1, True, False, "bf16", 128), (5, 3, 3, 256, 256, 3, False, True, "bf16", 256),
    (9, 6, 2, 128, 0, 1, True, False, "bf16", 16), (300, 24, 8, 64, 48, 2, False, False, "f32", 16),
    (2, 9, 1, 256, 16, 4, True, False, "f32", 16), (1500, 10, 2, 128, 128, 3, True, False, "bf16", 16),
])
def test_matches(sv, rows, Hq, Hkv, D, R, axes, norm, inter, dt, page):
    d = dev()
    rng = np.random.default_rng(rows * 1000 + D)
    total = Hq + 2 * Hkv
    x = torch.from_numpy(rng.normal(size=(rows, total, D)).astype(np.float32)).to(d)
    if dt == "bf16":
        x = x.bfloat16()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]  # slices of one buffer
    pages = -(-rows // page) + 2
    slots = rng.permutation(pages * page)[:rows].astype(np.int32)
    if rows > 2:
        slots[1], slots[2] = -1, pages * page  # both write nothing
    far = 2 ** 31 - 1 if rows % 2 else 1000
    pos = rng.integers(0, far, (rows, axes)).astype(np.int32)
    if rows > 4:
        pos[4] = -pos[4]
    inv = 1e6 ** (-np.arange(R // 2) / max(R // 2, 1))
    axis = rng.integers(0, axes, R // 2).astype(np.uint8)
    qw, kw = rng.normal(1, 0.2, D).astype(np.float32), rng.normal(1, 0.2, D).astype(np.float32)
    kc = torch.full((pages, Hkv, page, D), 7.0, dtype=torch.bfloat16, device=d)
    vc = torch.full((pages, Hkv, page, D), 9.0, dtype=torch.bfloat16, device=d)
    pt = torch.from_numpy(pos if axes > 1 else pos[:, 0]).contiguous().to(d)
    got = sv.rope_kv_append(
        q, k, v, pt, torch.from_numpy(slots).to(d),
        sv.rope_freqs(torch.from_numpy(inv).to(d)) if R else None, kc, vc,
        axis=torch.from_numpy(axis).to(d) if axes > 1 and R else None,
        q_weight=torch.from_numpy(qw).to(d) if norm else None,
        k_weight=torch.from_numpy(kw).to(d) if norm else None, interleaved=inter)
    xs = [t.double().cpu().numpy() for t in (q, k, v)]
    ax = axis if axes > 1 else None
    # the frequency the operator was given, from its words
    want_q, mag_q = ref.rotate(xs[0], pos, inv, ax, qw if norm else None, interleaved=inter)
    want_k, mag_k = ref.rotate(xs[1], pos, inv, ax, kw if norm else None, interleaved=inter)
    if far > 1000:  # a double's angle at 2^31 is itself off by up to 2^-22: allow for it
        mag_q, mag_k = 2 * mag_q, 2 * mag_k
    _close(got.double().cpu().numpy(), want_q, mag_q)
    kg, vg = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    seen = np.zeros((pages, page), bool)
    for r in range(rows):
        if not 0 <= slots[r] < pages * page:
            continue
        p, o = slots[r] // page, slots[r] % page
        seen[p, o] = True
        _close(kg[p, :, o], want_k[r], mag_k[r])
    ok = (slots >= 0) & (slots < pages * page)
    vref = v.bfloat16().double().cpu().numpy()
    assert np.array_equal(vg[slots[ok] // page, :, slots[ok] % page], vref[ok])
    assert (kg.transpose(0, 2, 1, 3)[~seen] == 7).all() and (vg.transpose(0, 2, 1, 3)[~seen] == 9).all()


def test_non_finite_values_stay_in_their_head(sv):
    d = dev()
    x = torch.randn(3, 6, 128, device=d)
    x[1, 0, 5], x[1, 2, 7], x[1, 4, 100] = float("nan"), float("inf"), float("-inf")
    kc = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16, device=d)
    vc = torch.zeros_like(kc)
    pos = torch.tensor([3, 4, 5], dtype=torch.int32, device=d)
    fr = sv.rope_freqs(torch.full((32,), 0.3, dtype=torch.float64, device=d))
    q = sv.rope_kv_append(x[:, :2], x[:, 2:4], x[:, 4:], pos, pos, fr, kc, vc)
    bad = ~torch.isfinite(q)
    assert bad[1, 0].sum() == 2 and bad.sum() == 2
    assert (~torch.isfinite(kc)).sum() == 2 and (~torch.isfinite(kc[0, 0, 4])).sum() == 2
    assert (~torch.isfinite(vc)).sum() == 1 and torch.isneginf(vc[0, 0, 4, 100])


def test_offsets_past_32_bits(sv):
    d = dev()
    pages, Hkv, page, D = 70000, 4, 64, 128  # 2.3e9 elements a cache
    kc = torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=d)
    vc = torch.zeros_like(kc)
    x = torch.randn(2, 12, D, device=d, dtype=torch.bfloat16)
    slots = torch.tensor([pages * page - 1, 64 * 65541 + 3], dtype=torch.int32, device=d)
    pos = torch.zeros(2, dtype=torch.int32, device=d)
    sv.rope_kv_append(x[:, :4], x[:, 4:8], x[:, 8:], pos, slots, None, kc, vc)
    for r, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, :, s % page], x[r, 4:8])
        assert torch.equal(vc[s // page, :, s % page], x[r, 8:])
    assert int(torch.count_nonzero(kc[0])) == 0
