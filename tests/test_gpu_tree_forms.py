"""paged_attn_tree's checks on the device and its masks, in each form of the kernels: what is
wrong with one request is flagged, shows in its outputs, and leaves the others as they were."""

from __future__ import annotations

import numpy as np
import pytest

import tree_ref as ref
from gpu_util import from_dev, to_dev, to_dev_i32
from test_gpu_tree_attn import Dev, gb  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# Hq, Hkv, D, Tn, cached tokens; the request at 1 is the one that goes wrong
FORMS = {
    "short": (8, 2, 128, 6, [40, 9, 0]),
    "whole, one row tile": (12, 2, 64, 12, [700, 300, 0]),
    "whole, two row tiles": (16, 2, 128, 20, [0, 300, 500]),
    "cut, one row tile": (12, 2, 128, 8, [3000, 2000, 20]),
    "cut, one row tile, D 64": (12, 2, 64, 8, [5000, 20, 1]),
    "cut, two row tiles": (16, 2, 64, 24, [3000, 1500, 20]),
    "teams": (32, 2, 128, 33, [2500, 900, 3]),
    "rounds of teams": (100, 1, 64, 20, [1500, 1000, 3]),
}


@pytest.fixture(params=FORMS.values(), ids=FORMS.keys())
def inputs(request):
    """Inputs whose table has a bound of 2000 tokens more than the caches hold."""
    c = ref.TreeInputs(*request.param, "random", None, 87000)
    extra = np.full((3, 125), -1, dtype=c.table.dtype)
    c.table = np.concatenate([c.table, extra], 1)
    return c, Dev(c)


def flags(gb):
    torch.cuda.synchronize()
    return gb.attn_device_status()[1]


def good_rows(c, o, lse, of):
    want, want_lse = of
    for r in (0, 2):
        assert torch.equal(o[r], want[r]) and torch.equal(lse[r], want_lse[r]), r


def test_as_given(gb, inputs):
    c, d = inputs
    o, lse = d.run(gb)
    assert flags(gb) == 0
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)


# the first number: tokens before the tree (None: as they are), the second: nodes
BAD = {"negative length": (-1, None), "most negative length": (-2 ** 31, None),
       "past the bound": ("bound", None), "length that wraps": (2 ** 31 - 2, None),
       "negative nodes": (None, -1), "most negative nodes": (None, -2 ** 31),
       "one node too many": (None, "many"), "nodes that wrap": (None, 2 ** 31 - 1)}


@pytest.mark.parametrize("bad", BAD.values(), ids=BAD.keys())
def test_bad_sizes(gb, inputs, bad):
    """The split of the work follows the lengths, so that the other requests' sums may be put
    together otherwise."""
    c, d = inputs
    Tn = c.q.shape[2]
    lens, nodes = d.lens.clone(), torch.full((3,), Tn, dtype=torch.int32, device="cuda")
    if bad[0] is not None:
        lens[1] = c.max_len - Tn + 1 if bad[0] == "bound" else bad[0]
    if bad[1] is not None:
        nodes[1] = Tn + 1 if bad[1] == "many" else bad[1]
    o, lse = d.run(gb, seq_lens=lens, tree_lens=nodes)
    assert flags(gb) == 2
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys, rows=[0, 2])
    d.run(gb)
    assert flags(gb) == 0


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("node,parent", [(0, 0), (3, 3), (5, -2), (2, 2 ** 31 - 1), (4, -2 ** 31), (5, 6)])
def test_bad_trees(gb, inputs, node, parent, ragged):
    c, d = inputs
    Tn = c.q.shape[2]
    n = Tn - (Tn > 6) if ragged else Tn
    nodes = to_dev_i32(np.array([Tn, n, Tn]))
    want = d.run(gb, tree_lens=nodes)
    parents = d.parents.clone()
    parents[1, node] = parent
    o, lse = d.run(gb, parents=parents, tree_lens=nodes)
    assert flags(gb) == (16 if node < n else 0)
    assert torch.isnan(o[1, :, :n]).all() and torch.isnan(lse[1, :, :n]).all()
    assert (o[1, :, n:] == 0).all() and torch.isneginf(lse[1, :, n:]).all()
    good_rows(c, o, lse, want)


def test_parents_behind_the_tree(gb, inputs):
    c, d = inputs
    Tn = c.q.shape[2]
    for n in ([Tn, 0, Tn], [Tn - 1, 2, 1]):
        nodes = to_dev_i32(np.array(n))
        want = d.run(gb, tree_lens=nodes)
        parents = d.parents.clone()
        for r, (k, x) in enumerate(zip(n, (99, -77, 2 ** 31 - 1))):
            parents[r, k:] = x
        o, lse = d.run(gb, parents=parents, tree_lens=nodes)
        assert flags(gb) == 0
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_bad_blocks(gb, inputs):
    c, d = inputs
    want = d.run(gb)
    last = (int(c.lens[1]) + c.q.shape[2] - 1) // 16
    for at in {0, last // 2, last}:
        for bad in (-1, -2 ** 31, c.k_pool.shape[0], 2 ** 31 - 1):
            table = d.table.clone()
            table[1, at] = bad
            o, lse = d.run(gb, block_table=table)
            assert flags(gb) == 4
            good_rows(c, o, lse, want)


def test_keys_that_are_not_seen(gb, inputs):
    """The key of a leaf may be infinite or NaN: no other node sees it."""
    c, d = inputs
    Tn = c.q.shape[2]
    c.parents[:, -1] = 0
    d = Dev(c)
    o, lse = d.run(gb)
    for bits in (0x7f80, 0xff80, 0x7fc0, 0x7f7f):
        k = c.k_pool.copy()
        for r, L in enumerate(c.lens):
            at = int(L) + Tn - 1
            k[c.table[r, at // 16], :, at % 16] = bits
        o2, lse2 = d.run(gb, k_pool=to_dev(k))
        assert torch.equal(o[:, :, :-1], o2[:, :, :-1]) and torch.equal(lse[:, :, :-1], lse2[:, :, :-1])
    assert flags(gb) == 0
