"""The compiled calls of gdn_inputs, gdn_advance and moe_smallm on tensors that cannot
be read: under a transform torch throws, and that has to reach Python as an exception,
not end the process.  Each case runs in a process of its own, on fake CUDA tensors (no
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
bf16, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

def make(*shape, dtype=bf16):
    return torch.empty(shape, dtype=dtype, device="cuda")

def four(n, k):
    return make(4, n, k // 8, dtype=i32), make(4, n, k // 64), make(4, n, k // 64)

first = {"gdn_inputs": (5, 96), "gdn_advance": (5, 2, 16), "moe_smallm": (5, 256)}

def call(name, x):
    if name == "gdn_inputs":
        args = (x, make(5, 4), make(5, 4), make(4, 96, dtype=f32), make(2, 3, 96, dtype=f32),
                make(4, dtype=f32), make(4, dtype=f32), make(3, dtype=i32), None, 3, True, 1.0, 1e-6,
                make(5, 2, 16), make(5, 2, 16), make(5, 4, 8), make(5, 4, dtype=f32),
                make(5, 4, dtype=f32))
    elif name == "gdn_advance":
        args = (x, make(5, 2, 16), make(5, 4, 8), make(5, 4, dtype=f32), make(5, 4, dtype=f32),
                make(2, 4, 8, 16, dtype=f32), make(3, dtype=i32), None, 3, make(5, 4, 8), None)
    else:
        args = (x, make(4, 256), *four(128, 256), *four(128, 256), *four(256, 128), 2, True,
                make(5, 256), None, None, make(1 << 20, dtype=u8))
    return getattr(calls, name)(0, 0, *args)

def raises(run):
    try:
        run()
    except RuntimeError as e:
        print("raised:", str(e).splitlines()[0])
        return
    raise SystemExit("nothing was raised")

name, how = {name!r}, {how!r}
with FakeTensorMode():
    x = make(3, *first[name])
    for _ in range(3):  # the process lives on: the call can be made again
        if how == "vmap":
            raises(lambda: torch.vmap(lambda x: call(name, x))(x))
        elif how == "grad":
            raises(lambda: torch.func.grad(lambda x: call(name, x))(x[0]))
        else:
            raises(lambda: torch.func.jvp(lambda x: call(name, x), (x[0],), (x[1],)))
    if how == "vmap":  # wrong kinds of arguments
        for args in ((), (0,), (0, 0, x[0]), (0, 0) + (x[0],) * 40):
            try:
                getattr(calls, name)(*args)
            except TypeError as e:
                print("refused:", e)
            else:
                raise SystemExit("%d arguments were taken" % len(args))
print("done")
"""


@pytest.mark.parametrize("how", ["vmap", "grad", "jvp"])
@pytest.mark.parametrize("name", ["gdn_inputs", "gdn_advance", "moe_smallm"])
def test_a_thrown_error_is_raised(name, how):
    code = SCRIPT.replace("{name!r}", repr(name)).replace("{how!r}", repr(how))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), (r.returncode, r.stdout, r.stderr[-800:])
