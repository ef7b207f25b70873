"""The example's attention layer through speculative cycles, against a dense
float64 recomputation of the last one."""
import sys
from pathlib import Path

import pytest

from gpu_util import sv_module

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cycles", [1, 7])
def test_attention_layer_through_cycles(cycles, capsys):
    sv_module()
    sys.path.insert(0, str(Path(__file__).resolve().parents[1] / "examples"))
    import attention_layer

    worst = attention_layer.main(["--cycles", str(cycles), "--check"])
    # queries, keys, values, weights and outputs are each rounded to bf16: the
    # half steps, 2^-8 each, add up in norm
    assert 0 < worst < 5 * 2.0 ** -8
    assert "flags [0, 0, 0, 0]" in capsys.readouterr().out
