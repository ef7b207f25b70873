"""gdn_inputs for every width of the convolution and every pair of types."""
import pytest
import torch

from gpu_util import sv_module
from test_gpu_gdn_rows import Layer, _check_inputs

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def sv():
    return sv_module()


@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("src", TYPES, ids=["from f32", "from bf16"])
@pytest.mark.parametrize("dst", TYPES, ids=["to f32", "to bf16"])
def test_every_width(sv, W, src, dst):
    """Sequences of every length up to the window's and one more (the next window
    keeps W - 1 - n of the old one's inputs), and one of three tiles."""
    c = Layer([*range(W + 1), 70], 2, 4, 128, 64, W, src, seed=50 + W)
    want = c.want(update=False)
    kept = c.window.clone()
    _check_inputs(c.run(sv, dtype=dst, update_window=False), c.window, want, dst, W)
    assert torch.equal(c.window, kept)
    want = c.want()
    _check_inputs(c.run(sv, dtype=dst), c.window, want, dst, W)


@pytest.mark.parametrize("W", [2, 5, 8])
def test_a_window_token_by_token_is_that_of_the_rows(sv, W):
    """Twelve rows at once, and one at a time."""
    whole, single = (Layer([12], 1, 2, 32, 32, W, torch.bfloat16, seed=60, pad=0) for _ in range(2))
    want = whole.run(sv)
    start = torch.tensor([0, 1], dtype=torch.int32, device=single.x.device)
    for t in range(12):
        got = sv.gdn_inputs(single.x[t:t + 1], single.a[t:t + 1], single.b[t:t + 1], single.weight,
                            single.window, single.a_log, single.dt, start, 1, k_heads=1, dk=32,
                            window_index=single.index)
        assert all(torch.equal(g[0], w[t]) for g, w in zip(got, want))
    assert torch.equal(single.window, whole.window)
