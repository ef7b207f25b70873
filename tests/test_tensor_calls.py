"""The compiled calls (csrc/tensors.cpp) on tensors that cannot be read: under a
transform torch throws, and that has to reach Python as an exception, not end
the process.  Each case runs in a process of its own, on fake CUDA tensors (no
GPU; the library is never reached)."""
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]

SCRIPT = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import mtp_speculative_decoding_qmv_gb300 as sv
from mtp_speculative_decoding_qmv_gb300 import build
build.build()
calls = sv._load_direct()

def make(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="cuda")

def call(name, x):
    i, bf16 = make, torch.bfloat16
    if name == "kv_pages_step":
        args = (x, i(2), i(2), i(4), i(2, 3), i(2), None, 0, 16, 2, i(2), i(2), i(2), i(3), i(2),
                i(2), i(2), i(2))
    elif name == "rope_kv_append":
        args = (x, i(3, 2, 64, dtype=bf16), i(3, 2, 64, dtype=bf16), i(3), i(3),
                i(8, dtype=torch.int64), i(2, 2, 16, 64, dtype=bf16), i(2, 2, 16, 64, dtype=bf16),
                None, None, None, 1e-6, False, i(3, 4, 64, dtype=bf16))
    else:
        args = (x, i(2, 2, 16, 64, dtype=bf16), i(2, 2, 16, 64, dtype=bf16), i(1, 2), i(2), i(1), 3,
                None, 0, i(3, 4, 64, dtype=bf16), None, i(1 << 20, dtype=torch.uint8))
    return getattr(calls, name)(0, 0, *args)

def raises(run):
    try:
        run()
    except RuntimeError as e:
        print("raised:", str(e).splitlines()[0])
        return
    raise SystemExit("nothing was raised")

name, how = {name!r}, {how!r}
first = (2,) if name == "kv_pages_step" else (3, 4, 64)
dtype = torch.int32 if name == "kv_pages_step" else torch.bfloat16
again = 3  # the process lives on and the lock is held: the call can be made again
with FakeTensorMode():
    x = make(5, *first, dtype=dtype)
    for _ in range(again):
        if how == "vmap":
            raises(lambda: torch.vmap(lambda x: call(name, x))(x))
        elif how == "grad":
            raises(lambda: torch.func.grad(lambda x: call(name, x))(x[0]))
        else:
            raises(lambda: torch.func.jvp(lambda x: call(name, x), (x[0],), (x[1],)))
print("done")
"""


@pytest.mark.parametrize("name,how", [
    ("kv_pages_step", "vmap"), ("rope_kv_append", "vmap"), ("rope_kv_append", "grad"),
    ("rope_kv_append", "jvp"), ("paged_attention", "vmap"), ("paged_attention", "grad"),
    ("paged_attention", "jvp")])
def test_a_thrown_error_is_raised(name, how):
    code = SCRIPT.replace("{name!r}", repr(name)).replace("{how!r}", repr(how))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), (r.returncode, r.stdout, r.stderr[-800:])
