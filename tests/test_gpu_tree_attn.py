"""paged_attn_tree against a plain implementation in 64 bits, and on the inputs where it could
go wrong."""

from __future__ import annotations

import numpy as np
import pytest

import tree_ref as ref
from gpu_util import from_dev, to_dev, to_dev_i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


class Dev:
    """TreeInputs on the GPU."""

    def __init__(self, c):
        self.c = c
        self.q, self.k, self.v = to_dev(c.q), to_dev(c.k_pool), to_dev(c.v_pool)
        self.table, self.lens = to_dev_i32(c.table), to_dev_i32(c.lens)
        self.parents = to_dev_i32(c.parents)
        self.nodes = to_dev_i32(c.nodes) if c.ragged else None

    def run(self, gb, **kw):
        a = dict(q=self.q, k_pool=self.k, v_pool=self.v, block_table=self.table,
                 seq_lens=self.lens, parents=self.parents, max_seq_len=self.c.max_len,
                 tree_lens=self.nodes, scale=self.c.scale)
        return gb.paged_attn_tree(**{**a, **kw})


CASES = [
    # Hq, Hkv, D, Tn, cached tokens, kind of tree, nodes
    (12, 2, 128, 8, [0, 1, 15, 16, 17, 120, 128, 513, 700], "random", None),
    (12, 2, 64, 8, [0, 1, 15, 16, 17, 120, 128, 513, 700], "random", None),
    (2, 2, 128, 1, [0, 1, 127, 128, 1000], "chain", None),          # decode's shape
    (5, 5, 64, 5, [3, 0, 260], "chain", None),
    (9, 3, 64, 37, [0, 5, 91, 400], "random", [0, 1, 37, 20]),
    (32, 1, 128, 4, [0, 2000, 300], "binary", None),                # 128 rows on a KV head
    (17, 1, 128, 8, [130, 0, 77], "random", None),                  # 136 rows: a second tile
    (64, 2, 128, 9, [0, 100, 1000], "random", [9, 0, 5]),           # 288 rows: a second pair
    (16, 1, 64, 64, [50, 0, 640, 127], "random", [64, 64, 1, 33]),  # 1024 rows
    (1, 1, 128, 256, [0, 1, 127, 128, 129, 500], "chain", None),    # the largest trees
    (2, 1, 64, 256, [0, 3, 250], "comb", [256, 200, 255]),
    (3, 3, 128, 130, [0, 126, 254, 1000], "star", [130, 129, 128, 127]),
    (4, 2, 128, 100, [2000, 28, 0, 29], "random", [0, 100, 0, 99]),
    (8, 4, 128, 33, [31, 95, 96, 4000], "binary", None),
    (128, 1, 64, 3, [70, 0, 2000], "random", [3, 0, 2]),            # a row tile a node
    (100, 1, 128, 20, [1500, 3], "random", [20, 7]),                # two rounds of teams
    (16, 16, 128, 1, [50, 700, 1], "chain", None),
    (6, 2, 128, 5, [700, 0, 64, 63], "comb", None),                 # 15 rows
    (8, 1, 64, 8, [1, 55, 56, 57, 120], "star", [8, 8, 8, 8, 8]),   # 64 rows
    (8, 2, 128, 8, [0, 60, 500, 330], "random", [8, 0, 5, 1]),      # 32 rows
]


@pytest.mark.parametrize("Hq,Hkv,D,Tn,lens,kind,nodes", CASES)
def test_matches_the_plain_form(gb, Hq, Hkv, D, Tn, lens, kind, nodes):
    c = ref.TreeInputs(Hq, Hkv, D, Tn, lens, kind, nodes, 70000 + Tn + D)
    o, lse = Dev(c).run(gb)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)


@pytest.mark.parametrize("Hq,Hkv,D,Tn,lens", [
    (8, 2, 128, 4, [9000, 3]),          # ranges that cut a cache many times
    (32, 8, 128, 32, [20000]),
    (4, 1, 64, 60, [15000, 0, 1]),      # 240 rows
    (40, 2, 64, 16, [5000, 4999, 1]),   # 320 rows
])
@pytest.mark.parametrize("slack", [0, 100000])
def test_long_caches(gb, Hq, Hkv, D, Tn, lens, slack):
    c = ref.TreeInputs(Hq, Hkv, D, Tn, lens, "random", None, 71000 + Tn, slack)
    d = Dev(c)
    o, lse = d.run(gb)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)
    o2, lse2 = d.run(gb)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_many_short_requests(gb):
    """More requests than the GPU has SMs, some empty."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 400).tolist()
    nodes = rng.integers(0, 7, 400).tolist()
    c = ref.TreeInputs(4, 2, 64, 6, lens, "random", nodes, 72000)
    o, lse = Dev(c).run(gb)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)


def test_a_chain_is_a_causal_chunk(gb):
    c = ref.TreeInputs(8, 2, 128, 40, [0, 10, 1000, 3001], "chain", None, 73000)
    d = Dev(c)
    o, lse = d.run(gb)
    o2, lse2 = gb.paged_attn_prefill(d.q, d.k, d.v, d.table, d.lens + 40, c.max_len, scale=c.scale)
    # both are within a bf16's half step for P and for O of the same values
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -6 * o2.float().abs().max()
    assert (lse - lse2).abs().max() <= 2.0 ** -16


def test_blocks_may_lie_anywhere(gb):
    c = ref.TreeInputs(12, 2, 128, 8, [700, 0, 3000], "random", None, 74000)
    d = Dev(c)
    o, lse = d.run(gb)
    NB = c.k_pool.shape[0]
    perm = torch.randperm(NB, generator=torch.Generator().manual_seed(1)).cuda()
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(NB, device="cuda")
    table = torch.where(d.table >= 0, inv[d.table.clamp(min=0).long()].int(), d.table)
    o2, lse2 = d.run(gb, k_pool=d.k[perm].contiguous(), v_pool=d.v[perm].contiguous(), block_table=table)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_large_scores_and_masked_infinities(gb):
    """A key that is not seen may be infinite or NaN; scores may be large."""
    c = ref.TreeInputs(4, 2, 128, 8, [40, 300], "binary", None, 75000)
    c.q = (c.q.astype(np.int32) + 0x0180).astype(np.uint16)  # times 8
    d = Dev(c)
    ref.check_attention(*map(from_dev, d.run(gb)), c.ref(), c.nodes, c.keys)
    # node 7 is a leaf: nobody else sees its key
    o, lse = d.run(gb)
    for bits in (0x7f80, 0xff80, 0x7fc0):
        k = c.k_pool.copy()
        for r, L in enumerate(c.lens):
            k[c.table[r, (L + 7) // 16], :, (L + 7) % 16] = bits
        o2, lse2 = d.run(gb, k_pool=to_dev(k))
        assert torch.equal(o[:, :, :7], o2[:, :, :7]) and torch.equal(lse[:, :, :7], lse2[:, :, :7])


def test_outputs_given_and_left_out(gb):
    c = ref.TreeInputs(4, 2, 64, 5, [33, 0, 4], "random", None, 76000)
    d = Dev(c)
    o, lse = d.run(gb)
    out, out_lse = torch.full_like(o, 7), torch.full_like(lse, 7)
    got = d.run(gb, out=out, lse=out_lse)
    assert got[0] is out and got[1] is out_lse and torch.equal(out, o) and torch.equal(out_lse, lse)
    o2, none = d.run(gb, return_lse=False)
    assert none is None and torch.equal(o2, o)
    empty = d.q[:, :, :0].contiguous()
    o3, lse3 = d.run(gb, q=empty, parents=d.parents[:, :0].contiguous())
    assert o3.shape == (3, 4, 0, 64) and lse3.shape == (3, 4, 0)


@pytest.mark.parametrize("lens,nodes", [([100, -1, 40], None), ([100, 5000, 40], None),
                                        ([100, 50, 40], [8, 9, 8]), ([100, 50, 40], [8, -1, 8]),
                                        ([100, 2 ** 31 - 4, 40], None)])
def test_bad_sizes_are_flagged(gb, lens, nodes):
    c = ref.TreeInputs(12, 2, 128, 8, [100, 50, 40], "random", None, 77000)
    d = Dev(c)
    o, lse = d.run(gb)
    n = None if nodes is None else to_dev_i32(np.array(nodes))
    o2, lse2 = d.run(gb, seq_lens=to_dev_i32(np.array(lens)), tree_lens=n)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2)
    assert torch.isnan(o2[1]).all() and torch.isnan(lse2[1]).all()
    ref.check_attention(from_dev(o2), from_dev(lse2), c.ref(), c.nodes, c.keys, rows=[0, 2])
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)


@pytest.mark.parametrize("node,parent", [(0, 0), (3, 3), (7, 100), (5, -2), (2, 6), (4, -2 ** 31)])
@pytest.mark.parametrize("L", [50, 2500])
def test_bad_trees_are_flagged(gb, node, parent, L):
    c = ref.TreeInputs(12, 2, 128, 8, [100, L, 40], "random", None, 78000)
    d = Dev(c)
    parents = d.parents.clone()
    parents[1, node] = parent
    o, lse = d.run(gb, parents=parents)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 16)
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys, rows=[0, 2])


def test_parents_behind_the_tree_are_not_read(gb):
    c = ref.TreeInputs(4, 2, 128, 8, [100, 50], "random", [5, 0], 78100)
    d = Dev(c)
    o, lse = d.run(gb)
    parents = d.parents.clone()
    parents[0, 5:] = 99
    parents[1] = -77
    o2, lse2 = d.run(gb, parents=parents)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)


def test_bad_blocks_are_flagged(gb):
    c = ref.TreeInputs(4, 2, 128, 8, [100, 50, 40], "random", None, 79000)
    d = Dev(c)
    for bad in (-1, c.k_pool.shape[0], 2 ** 31 - 1):
        table = d.table.clone()
        table[1, 2] = bad
        o, lse = d.run(gb, block_table=table)
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 4)
        ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys, rows=[0, 2])


def test_side_stream_and_workspace(gb):
    c = ref.TreeInputs(12, 2, 128, 8, [3000, 10, 2000], "random", None, 80000)
    d = Dev(c)
    o, lse = d.run(gb)
    need = gb.paged_attn_tree_workspace_size(3, 8, 12, 2, 128, c.max_len)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = d.run(gb, stream=s)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")  # NaNs
    o3, lse3 = d.run(gb, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)
    if need:
        with pytest.raises(gb.GbAttnError):
            d.run(gb, workspace=ws[:need - 1])


def test_outputs_are_written_nowhere_else(gb):
    c = ref.TreeInputs(9, 3, 64, 37, [0, 5, 91, 1400], "random", [0, 1, 37, 20], 81000)
    d = Dev(c)
    o, lse = d.run(gb)
    pad = 4096
    big = torch.full((o.numel() + 2 * pad,), 3, dtype=torch.bfloat16, device="cuda")
    big_l = torch.full((lse.numel() + 2 * pad,), 3, dtype=torch.float32, device="cuda")
    need = gb.paged_attn_tree_workspace_size(4, 37, 9, 3, 64, c.max_len)
    ws = torch.full((need + 2 * pad,), 17, dtype=torch.uint8, device="cuda")
    d.run(gb, out=big[pad:-pad].view(o.shape), lse=big_l[pad:-pad].view(lse.shape),
          workspace=ws[pad:pad + need] if need else None)
    torch.cuda.synchronize()
    assert torch.equal(big[pad:-pad].view(o.shape), o) and torch.equal(big_l[pad:-pad].view(lse.shape), lse)
    for t, v in ((big, 3), (big_l, 3)):
        assert (t[:pad] == v).all() and (t[-pad:] == v).all()
    assert (ws[:pad] == 17).all() and (ws[pad + need:] == 17).all()


def test_graph_replays_follow_the_lengths(gb):
    c = ref.TreeInputs(12, 2, 128, 8, [700, 20, 3000], "random", [8, 5, 7], 82000)
    d = Dev(c)
    o, lse = d.run(gb)
    less = torch.tensor([100, 20, 2999], dtype=torch.int32, device="cuda")
    o_less, lse_less = d.run(gb, seq_lens=less)
    lens = d.lens.clone()
    out, out_lse = torch.empty_like(o), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run(gb, seq_lens=lens, out=out, lse=out_lse)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(out_lse, lse)
        lens.copy_(less)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o_less) and torch.equal(out_lse, lse_less)
        lens.copy_(d.lens)


# short caches, whole segments, segments cut between CTAs
KINDS = [(8, 2, 128, 6, [0, 5, 40]), (16, 2, 64, 20, [0, 300, 500]), (12, 2, 128, 8, [3000, 20]),
         (32, 2, 128, 33, [2500, 3, 900])]


@pytest.mark.parametrize("Hq,Hkv,D,Tn,lens", KINDS)
@pytest.mark.parametrize("scale", [1e-38, 1e-6, 1.0, 3.0])
def test_softmax_scales(gb, Hq, Hkv, D, Tn, lens, scale):
    c = ref.TreeInputs(Hq, Hkv, D, Tn, lens, "random", None, 83000)
    c.scale = scale
    o, lse = Dev(c).run(gb)
    torch.cuda.synchronize()
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)


def test_more_requests_than_threads(gb):
    """Ranges of a batch of more requests than a CTA has threads, some without nodes."""
    rng = np.random.default_rng(6)
    lens, nodes = rng.integers(0, 1500, 900).tolist(), rng.integers(0, 4, 900).tolist()
    c = ref.TreeInputs(2, 1, 64, 3, lens, "random", nodes, 84000, slack=3000)
    o, lse = Dev(c).run(gb)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)


@pytest.mark.parametrize("Hq,Hkv,D,Tn,lens", KINDS)
def test_the_loosest_bound_on_the_lengths(gb, Hq, Hkv, D, Tn, lens):
    c = ref.TreeInputs(Hq, Hkv, D, Tn, lens[:1], "random", None, 85000)
    o, lse = Dev(c).run(gb, max_seq_len=2 ** 31 - 1)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    ref.check_attention(from_dev(o), from_dev(lse), c.ref(), c.nodes, c.keys)


def test_calls_on_two_streams_and_a_graph_at_once(gb):
    cs = [Dev(ref.TreeInputs(*k, "random", None, 86000 + i)) for i, k in enumerate(KINDS)]
    want = [d.run(gb) for d in cs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [d.run(gb) for d in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        with torch.cuda.stream(streams[2]):
            graph.replay()
        for s in (0, 1):
            for d in (cs, cs[::-1])[s]:
                got[s].append(d.run(gb, stream=streams[s]))
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    n = len(cs)
    for i, (o, lse) in enumerate(want):
        for o2, lse2 in got[0][i::n] + got[1][n - 1 - i::n] + [captured[i]]:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
