"""moe_smallm's outputs are fp32 results rounded once."""
import pytest
import torch

import moe_rounding as ref
import rounding
from gpu_util import sv_module
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    return sv_module()


def _host(m):
    return m[0].cpu().numpy(), m[1].double().cpu().numpy(), m[2].double().cpu().numpy()


def _faults(c, y, **kw):
    want, err, _ = ref.layer(c.x.double().cpu().numpy(), c.router.double().cpu().numpy(), _host(c.gate),
                             _host(c.up), _host(c.down), c.sizes[4], ids=c.ids.cpu().numpy(), **kw)
    return rounding.faults(y.double().cpu().numpy(), want, err)


@pytest.mark.parametrize("rows,hidden,inter,experts,top", [
    (1, 2048, 512, 32, 8), (2, 65536, 128, 3, 2), (3, 2560, 1024, 40, 5), (4, 5120, 1024, 8, 6), (9, 256, 256, 3, 1),
    (19, 2560, 896, 12, 4), (33, 512, 384, 5, 2), (64, 1024, 640, 16, 4), (128, 2048, 1024, 12, 2),
    (128, 1024, 256, 32, 4)])
def test_outputs_are_rounded_once(sv, rows, hidden, inter, experts, top):
    c = Layer(rows, hidden, inter, experts, top, seed=41)
    fault = _faults(c, c.run(sv))
    assert not fault, fault
    sv.device_status()


def test_softmax_over_all_experts(sv):
    c = Layer(17, 1024, 256, 16, 4, seed=42)
    fault = _faults(c, c.run(sv, renormalize=False), renormalize=False)
    assert not fault, fault


@pytest.mark.parametrize("power", [-100, -30, 40, 100])
def test_inputs_of_any_size(sv, power):
    """x times a power of two, gate's weights by its inverse: silu sees what it saw."""
    c = Layer(9, 512, 256, 4, 2, seed=43)
    y = c.run(sv)
    want = c.ids.clone()
    c.x *= 2.0 ** power
    c.router *= 2.0 ** -power
    c.gate = (c.gate[0], c.gate[1] * 2.0 ** -power, c.gate[2] * 2.0 ** -power)
    c.up = (c.up[0], c.up[1] * 2.0 ** -power, c.up[2] * 2.0 ** -power)
    assert torch.equal(c.run(sv), y) and torch.equal(c.ids, want)
