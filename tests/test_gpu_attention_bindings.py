"""What the paged cache's three calls refuse of their tensors: each by its own
error, before anything is launched."""
import pytest
import torch

from gpu_util import sv_module

pytestmark = pytest.mark.gpu
I32, BF16, F32 = torch.int32, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def ints(*shape):
    return torch.zeros(shape, dtype=I32, device="cuda")


def rows(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def pages_args():
    return dict(length=ints(2), held=ints(2), cursor=torch.tensor([0, 4], dtype=I32, device="cuda"),
                ring=torch.arange(4, dtype=I32, device="cuda"), block_table=ints(2, 3),
                n_new=ints(2) + 1, page_size=16, rows=2)


def append_args():
    return dict(q=rows(3, 4, 64), k=rows(3, 2, 64), v=rows(3, 2, 64), positions=ints(3),
                slots=ints(3), freqs=torch.zeros(8, dtype=torch.int64, device="cuda"),
                k_cache=rows(2, 2, 16, 64), v_cache=rows(2, 2, 16, 64))


def attend_args(sv):
    return dict(q=rows(3, 4, 64), k_cache=rows(2, 2, 16, 64), v_cache=rows(2, 2, 16, 64),
                block_table=ints(1, 2), q_start=torch.tensor([0, 3], dtype=I32, device="cuda"),
                kv_len=ints(1) + 3, max_new=3, workspace=sv.make_attention_workspace(64, "cuda"))


def refused(fn, args, error, **changed):
    with pytest.raises(error):
        fn(**{**args, **changed})
    torch.cuda.synchronize()


@pytest.mark.parametrize("changed,error", [
    (dict(held=lambda: ints(3)), ValueError),
    (dict(held=lambda: ints(2).long()), TypeError),
    (dict(held=lambda: ints(2).cpu()), ValueError),
    (dict(n_new=lambda: ints(4)[::2]), ValueError),
    (dict(n_new=lambda: [1, 1]), TypeError),
    (dict(n_commit=lambda: ints(2).float()), TypeError),
    (dict(slots=lambda: ints(3)), ValueError),
    (dict(cursor=lambda: ints(1)), ValueError),
    (dict(rows=lambda: 1 << 31), (OverflowError, RuntimeError)),
    (dict(n_commit_bias=lambda: 1 << 32), OverflowError),
    (dict(page_size=lambda: (1 << 32) + 16), OverflowError),
])
def test_kv_pages_step(sv, changed, error):
    args, changed = pages_args(), {k: f() for k, f in changed.items()}
    if "rows" in changed:  # outputs of the right length cannot be had: give some
        changed.update(slots=ints(2), positions=ints(2), length_out=ints(2), held_out=ints(2),
                       cursor_out=ints(2), q_start=ints(3), kv_len=ints(2), err_flags=ints(2))
    refused(sv.kv_pages_step, args, error, **changed)
    step = sv.kv_pages_step(**args)
    assert step.kv_len.tolist() == [1, 1] and step.err_flags.tolist() == [0, 0]


@pytest.mark.parametrize("changed,error", [
    (dict(q=lambda: rows(3, 4, 64, dtype=torch.float16)), TypeError),
    (dict(q=lambda: rows(3, 4, 64, dtype=F32)), TypeError),  # k and v are bf16
    (dict(k=lambda: rows(3, 3, 64)), ValueError),
    (dict(v=lambda: rows(3, 2, 128)[..., ::2]), ValueError),
    (dict(v=lambda: rows(2, 3, 64).transpose(0, 1)), ValueError),
    (dict(v=lambda: rows(3, 2, 64).cpu()), ValueError),
    (dict(positions=lambda: ints(2)), ValueError),
    (dict(positions=lambda: ints(3).long()), TypeError),
    (dict(slots=lambda: ints(3, 1)), ValueError),
    (dict(freqs=lambda: torch.zeros(2, 4, dtype=torch.int64, device="cuda")), ValueError),
    (dict(freqs=lambda: rows(8, dtype=torch.float64)), TypeError),
    (dict(axis=lambda: torch.zeros(7, dtype=torch.uint8, device="cuda")), ValueError),
    (dict(q_weight=lambda: rows(64)), TypeError),
    (dict(k_weight=lambda: rows(32, dtype=F32)), ValueError),
    (dict(v_cache=lambda: rows(3, 2, 16, 64)), ValueError),
    (dict(q_out=lambda: rows(3, 4, 64, dtype=F32)), TypeError),
])
def test_rope_kv_append(sv, changed, error):
    args = append_args()
    args["k_cache"].fill_(7.0)
    refused(sv.rope_kv_append, args, error, **{k: f() for k, f in changed.items()})
    assert (args["k_cache"] == 7.0).all()
    assert sv.rope_kv_append(**args).shape == (3, 4, 64)


@pytest.mark.parametrize("changed,error", [
    (dict(q=lambda: rows(3, 4, 64, dtype=F32)), TypeError),
    (dict(q=lambda: rows(3, 4, 128)[..., ::2]), ValueError),
    (dict(v_cache=lambda: rows(2, 2, 32, 64)), ValueError),
    (dict(block_table=lambda: ints(2)), ValueError),
    (dict(block_table=lambda: ints(1, 4)[:, ::2]), ValueError),
    (dict(q_start=lambda: ints(3)), ValueError),
    (dict(kv_len=lambda: ints(1).long()), TypeError),
    (dict(out=lambda: rows(3, 4, 64, dtype=F32)), TypeError),
    (dict(out=lambda: rows(2, 4, 64)), ValueError),
    (dict(lse=lambda: rows(3, 4)), TypeError),
    (dict(lse=lambda: rows(4, 4, dtype=F32)), ValueError),
    (dict(workspace=lambda: torch.zeros(4096, device="cuda")), TypeError),
    (dict(workspace=lambda: torch.zeros(4096, dtype=torch.uint8, device="cuda")), RuntimeError),
    (dict(window=lambda: 1 << 32), OverflowError),
    (dict(max_new=lambda: 1 << 32), OverflowError),
])
def test_paged_attention(sv, changed, error):
    args = attend_args(sv)
    refused(sv.paged_attention, args, error, **{k: f() for k, f in changed.items()})
    out, lse = sv.paged_attention(**args)
    assert lse is None and (out == 0).all()
