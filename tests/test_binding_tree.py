"""The compiled binding of the operators for trees of drafted tokens and tensors without memory
(test_binding_transforms.py says why): what a function transform hands over is left to the
Python wrappers, as is every call that is not the usual one.  No GPU is needed: the tensors are
fake ones on a CUDA device, each case is a child process."""

from __future__ import annotations

import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

CHILD = """
import ctypes, importlib, sys
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import attention_flashattention_fwd_03_gb300 as gb

transform = sys.argv[1]
try:
    m = importlib.import_module("._binding", gb.__name__)
except ImportError:
    print("not built")
    sys.exit()
gb._load_torch()
h = gb.lib()
first = ("qkv_norm_rope", "qkv_norm_rope_bwd", "qkv_norm_rope_bwd_workspace_size",
         "paged_qkv_append", "paged_kv4_append", "paged_kv4_gather", "paged_kv4_attn_decode",
         "paged_kv4_attn_decode_workspace_size", "paged_kv4_attn_prefill",
         "paged_kv4_attn_prefill_workspace_size")
names = ("paged_attn_tree", "paged_attn_tree_workspace_size", "draft_verify", "paged_kv_keep")
address = lambda n: ctypes.cast(getattr(h, n), ctypes.c_void_p).value
m.setup(torch.__version__, lambda: 0, lambda d: 0, *map(address, first))
m.setup_tree(*map(address, names))
for wrong in ((), (1, 2, 3), (1, 2, 3, 4, 5)):
    try:
        m.setup_tree(*wrong)
    except TypeError:
        continue
    raise AssertionError(wrong)

bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
q, pool = ((3, 4, 5, 64), bf16), ((9, 2, 16, 64), bf16)
table, lens, nodes = ((3, 2), i32), ((3,), i32), ((3, 5), i32)
probs = ((3, 5, 70), f32)
calls = dict(
    tree=[q, pool, pool, table, lens, nodes, 32, lens, None, q, ((3, 4, 5), f32), None, True],
    verify=[probs, probs, nodes, nodes, ((3, 5), f32), lens, nodes, nodes, lens],
    keep=[pool, pool, table, lens, nodes, lens, lens],
)


class Enough(Exception):  # ends a transform after its call (its gradients would need a GPU)
    pass


seen = []
with FakeTensorMode():
    for entry, args in calls.items():
        at = [i for i, a in enumerate(args) if isinstance(a, tuple)]

        def record(*tensors):
            full = list(args)
            for i, t in zip(at, tensors):
                full[i] = t
            seen.append(getattr(m, entry)(*full))
            raise Enough

        batch = (2,) if transform == "vmap" else ()
        made = [torch.empty(batch + args[i][0], dtype=args[i][1], device="cuda") for i in at]
        if transform == "unusual":  # wrong types, sizes, counts of arguments, devices
            good = list(args)
            for i, t in zip(at, made):
                good[i] = t
            for i in at:
                for bad in (None if entry != "tree" else 7, good[i].double(), good[i][..., :-1], "x",
                            torch.empty(args[i][0], dtype=args[i][1])):
                    if bad is None and (entry, i) in (("verify", 1), ("verify", 5), ("verify", 6),
                                                      ("verify", 7), ("verify", 8), ("keep", 6)):
                        continue
                    seen.append(getattr(m, entry)(*good[:i], bad, *good[i + 1:]))
            seen.append(getattr(m, entry)(*good[:-1]))
            continue
        try:
            if transform == "vmap":
                torch.func.vmap(record)(*made)
            else:
                torch.func.grad(record, argnums=0)(*made)
        except Enough:
            pass
assert seen == [None] * len(seen) and len(seen) >= len(calls), seen
print("left to the wrapper")
"""


@pytest.mark.parametrize("transform", ["vmap", "grad", "unusual"])
def test_unusual_tensors_are_left_to_the_wrapper(transform):
    r = subprocess.run([sys.executable, "-c", CHILD, transform], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr[-2000:])
    if "not built" in r.stdout:
        pytest.skip("_binding was not built")
    assert "left to the wrapper" in r.stdout, r.stderr[-2000:]
