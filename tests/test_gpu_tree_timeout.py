"""The bounded waits of paged_attn_tree's kernels, as in test_gpu_timeout.py: their copy warps
withhold their first copy, the waiting roles give up after a millisecond, the flag is
reported, and the next call is right."""

from __future__ import annotations

import pytest

import tree_ref as ref
from gpu_util import from_dev
from test_gpu_timeout import _with_short_limit
from test_gpu_tree_attn import Dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


@pytest.mark.parametrize("Hq,Hkv,D,Tn,lens", [
    (12, 2, 128, 4, [100, 0, 300]),           # small trees over short caches
    (12, 2, 128, 30, [100, 0, 300]),          # whole segments, two row tiles
    (12, 2, 128, 8, [3000, 900, 5000]),       # cut segments, one row tile
    (32, 2, 64, 100, [3000, 900]),            # teams
])
def test_a_wait_that_runs_out_is_reported(gb, Hq, Hkv, D, Tn, lens):
    c = ref.TreeInputs(Hq, Hkv, D, Tn, lens, "random", None, 83000 + Tn)
    d = Dev(c)
    need = gb.paged_attn_tree_workspace_size(len(lens), Tn, Hq, Hkv, D, c.max_len)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    st, flags = _with_short_limit(gb, lambda: d.run(gb, workspace=ws))
    assert st == gb.ATTN_ERR_DEVICE and flags & 1, (st, flags)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    o, lse = d.run(gb)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)
