"""The compiled binding and tensors that have no memory: what torch.func's transforms hand
to a function is a plain torch.Tensor on a CUDA device by its type and attributes, but a
wrapper without storage.  The binding leaves such calls to the Python wrappers (whose
error names the reason) in whichever thread they are made.

No GPU is needed: the tensors are fake ones on a CUDA device, wrapped by a transform, and
the current device and stream are stand-ins.  Each case is a child process, so that one
that ends its process is a failed test.
"""

from __future__ import annotations

import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

CHILD = """
import ctypes, importlib, sys, threading
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import attention_flashattention_fwd_03_gb300 as gb

transform, where = sys.argv[1:]
try:
    m = importlib.import_module("._binding", gb.__name__)
except ImportError:
    print("not built")
    sys.exit()
names = ("qkv_norm_rope", "qkv_norm_rope_bwd", "qkv_norm_rope_bwd_workspace_size",
         "paged_qkv_append", "paged_kv4_append", "paged_kv4_gather", "paged_kv4_attn_decode",
         "paged_kv4_attn_decode_workspace_size", "paged_kv4_attn_prefill",
         "paged_kv4_attn_prefill_workspace_size")
h = gb.lib()
m.setup(torch.__version__, lambda: 0, lambda d: 0,
        *(ctypes.cast(getattr(h, n), ctypes.c_void_p).value for n in names))


bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
rows, heads = ((3, 4, 5, 64), bf16), ((3, 5, 4, 64), bf16)
paged = [((3, 2), i32), ((3,), i32)]
norm = [None, None, None, 1e-6, False, None]  # cos_sin, weights, eps, interleaved, positions
pool = ((9, 5, 18 * 64), u8)
calls = dict(
    rope=[rows, rows, rows, *norm, heads, heads, heads],
    rope_bwd=[heads, heads, heads, rows, rows, *norm],
    append=[rows, rows, rows, *[((9, 5, 16, 64), bf16)] * 2, *paged, *norm, heads, ((3,), i32)],
    append4=[rows, rows, rows, pool, None, *paged, *norm, heads, ((3,), i32)],
    gather=[pool, *paged, 7, *[((3, 5, 7, 64), bf16)] * 2],
    decode=[((3, 5, 64), bf16), pool, *paged, 32, None, ((3, 5, 64), bf16), ((3, 5), torch.float32),
            None, True],
    prefill=[heads, pool, *paged, 32, None, heads, ((3, 5, 4), torch.float32), None, True, True],
)


class Enough(Exception):  # ends a transform after its call (its gradients would need a GPU)
    pass


def leave(entry, args):
    at = [i for i, a in enumerate(args) if isinstance(a, tuple)]

    def record(*tensors):
        full = list(args)
        for i, t in zip(at, tensors):
            assert type(t) is torch.Tensor and t.is_cuda and t.shape == args[i][0]
            full[i] = t
        seen.append(getattr(m, entry)(*full))
        raise Enough

    batch = (2,) if transform == "vmap" else ()
    made = [torch.empty(batch + args[i][0], dtype=args[i][1], device="cuda") for i in at]
    try:
        if transform == "vmap":
            torch.func.vmap(record)(*made)
        else:  # (of a floating-point operand, which not every first one is)
            n = next(i for i, t in enumerate(made) if t.is_floating_point())
            torch.func.grad(record, argnums=n)(*made)
    except Enough:
        pass


def run():
    with FakeTensorMode():
        for entry, args in calls.items():
            print(entry, flush=True)
            leave(entry, args)


seen = []
if where == "thread":
    t = threading.Thread(target=run)
    t.start()
    t.join()
else:
    run()
assert seen == [None] * len(calls), seen
print("left to the wrapper")
"""


@pytest.mark.parametrize("where", ["here", "thread"])
@pytest.mark.parametrize("transform", ["vmap", "grad"])
def test_wrapped_tensors_are_left_to_the_wrapper(transform, where):
    r = subprocess.run([sys.executable, "-c", CHILD, transform, where], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr[-2000:])
    if "not built" in r.stdout:
        pytest.skip("_binding was not built")
    assert "left to the wrapper" in r.stdout, r.stderr[-2000:]
