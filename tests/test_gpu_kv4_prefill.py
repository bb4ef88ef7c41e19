"""paged_kv4_attn_prefill against the bf16 paged prefill over the same values (equal bits:
every value the 4-bit cache holds is a bf16) and against the fp64 oracle."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import rope_ref as ref
import synth
from gpu_util import check_close, from_dev, to_dev, to_dev_i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


class Item:
    def __init__(self, Hq, Hkv, D, Tq, lens, seed):
        cfg = synth.DecodeConfig("kv4p", len(lens), Hq, Hkv, D, 0, 1, 16, seed)
        p = synth.paged_inputs(cfg, seq_lens=lens, max_seq_len=max(max(lens), 1))
        self.p, self.scale, self.lens = p, cfg.softmax_scale, lens
        self.q_bits = synth.normal_bf16(seed + 11, (len(lens), Hq, Tq, D))
        self.q = to_dev(self.q_bits)
        self.pool_host = ref.pool_from_bf16(p.k_pool, p.v_pool)  # dead slots: NaN scales
        self.k, self.v = ref.value_bits(p.k_pool), ref.value_bits(p.v_pool)
        self.pool = torch.from_numpy(self.pool_host).cuda()
        self.table, self.kv_lens = to_dev_i32(p.block_table), to_dev_i32(p.seq_lens)

    def run(self, gb, causal, **kw):
        return gb.paged_kv4_attn_prefill(self.q, kw.pop("pool", self.pool), kw.pop("table", self.table),
                                         kw.pop("lens", self.kv_lens), self.p.max_seq_len,
                                         causal=causal, scale=self.scale, **kw)


CASES = [
    # Hq, Hkv, D, Tq, kv_lens
    (8, 2, 128, 1, [1, 17, 4096, 8192]),
    (8, 2, 128, 127, [127, 300, 2049, 8192]),
    (8, 2, 128, 512, [512, 700, 5000, 8192]),
    (12, 2, 128, 300, [300, 301, 1024, 2999]),
    (4, 4, 64, 257, [257, 640, 1000, 4096]),
    (16, 2, 64, 512, [600, 8192]),
    (2, 1, 128, 37, [0, 5, 36, 37, 128, 129]),   # chunks longer than their cache
    (2, 1, 64, 130, [0, 1, 15, 16, 17, 127]),
]


@pytest.mark.parametrize("Hq,Hkv,D,Tq,lens", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_equals_the_bf16_prefill_over_the_same_values(gb, Hq, Hkv, D, Tq, lens, causal):
    c = Item(Hq, Hkv, D, Tq, lens, 60000 + Tq)
    o, lse = c.run(gb, causal)
    o2, lse2 = gb.paged_attn_prefill(c.q, to_dev(c.k), to_dev(c.v), c.table, c.kv_lens,
                                     c.p.max_seq_len, causal=causal, scale=c.scale)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,Hkv,D,Tq,lens", [CASES[3], CASES[4], CASES[6], CASES[7]])
def test_matches_the_oracle(gb, Hq, Hkv, D, Tq, lens):
    c = Item(Hq, Hkv, D, Tq, lens, 61000 + Tq)
    o, lse = c.run(gb, True)
    o_ref, l_ref = oracle.paged_prefill(c.q_bits, c.k, c.v, c.p.block_table, c.p.seq_lens, True,
                                        c.scale)
    og, lg = from_dev(o), from_dev(lse)
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lg), empty) and np.all(og[empty] == 0)
    check_close(og[~empty], lg[~empty], o_ref[~empty], l_ref[~empty], "kv4 prefill")


def test_outputs_streams_and_graphs(gb):
    c = Item(8, 2, 128, 130, [130, 999, 2048], 62000)
    o, lse = c.run(gb, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, none = c.run(gb, True, return_lse=False, stream=s)
    s.synchronize()
    assert none is None and torch.equal(o, o2)
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(gb, True, out=out, lse=l2)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(l2, lse)


def test_nan_keys_reach_the_queries_that_see_them(gb):
    Tq, D = 20, 128
    c = Item(4, 2, D, Tq, [40, 40], 63000)
    host = c.pool_host.copy()
    blk = c.p.block_table
    # token 30 of item 0: its key in head 0 (seen by queries 10..19)
    host[blk[0, 1], 0, 8 * D + 14 * 8:8 * D + 14 * 8 + 2] = [0xC0, 0x7F]
    o, lse = c.run(gb, True, pool=torch.from_numpy(host).cuda())
    good, _ = c.run(gb, True)
    nan = torch.isnan(lse).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, :2, 10:] = True
    assert np.array_equal(nan, want)
    assert np.array_equal(torch.isnan(o).all(-1).cpu().numpy(), want)
    keep = torch.from_numpy(~want).cuda()
    assert torch.equal(o[keep], good[keep])


def test_bad_requests_are_flagged(gb):
    c = Item(4, 2, 64, 30, [100, 200, 300, 100], 64000)
    table = c.p.block_table.copy()
    table[1, 5] = c.p.num_pool_blocks
    lens = c.p.seq_lens.copy()
    lens[2], lens[3] = 301, -1
    o, lse = c.run(gb, True, table=to_dev_i32(table), lens=to_dev_i32(lens))
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2 | 4)
    assert torch.isnan(o[2:]).all() and torch.isnan(lse[2:]).all()
    good, _ = c.run(gb, True)
    assert torch.equal(o[0], good[0])  # item 1 read another block: unspecified


def test_a_wait_that_runs_out_is_reported(gb):
    c = Item(4, 2, 128, 30, [100, 200], 65000)
    gb.test_set_failure(2_000_000, True)
    try:
        c.run(gb, True)
        torch.cuda.synchronize()
        st, flags = gb.attn_device_status()
    finally:
        gb.test_set_failure(0, False)
    assert st == gb.ATTN_ERR_DEVICE and flags & 1
    o, lse = c.run(gb, True)
    o2, _ = c.run(gb, True)
    assert torch.equal(o, o2) and gb.attn_device_status() == (gb.ATTN_OK, 0)


def test_a_prompt_in_chunks_then_decode(gb):
    """A prompt through the whole path in two chunks and one token more -- projection
    rows, norm, rotation, quantised append, attention -- equals the prompt in one chunk."""
    Hq, Hkv, D, T = 8, 2, 128, 200
    rows = to_dev(synth.normal_bf16(66000, (2, T + 1, Hq + 2 * Hkv, D)))
    cs = torch.from_numpy(ref.table(T + 1, D)).cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    table = to_dev_i32(synth.permutation(9, 28).reshape(2, 14))

    def run(cuts):
        pool = torch.zeros((28, Hkv, 18 * D), dtype=torch.uint8, device="cuda")
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        out = []
        for a, b in zip(cuts, cuts[1:]):
            q, k, v = rows[:, a:b].split([Hq, Hkv, Hkv], 2)
            new = torch.empty_like(lens)
            q, _ = gb.paged_kv4_append(q, k, v, pool, table, lens, cs, w, w, new_seq_lens=new)
            o, lse = gb.paged_kv4_attn_prefill(q, pool, table, new, T + 1)
            if b - a == 1:
                o1, lse1 = gb.paged_kv4_attn_decode(q.squeeze(2), pool, table, new, T + 1)
                # the two kernels round probabilities at different points: half a step
                # of 2^-8 of sum p |v| each, |v| being at most 5.3 here
                assert torch.all((o1 - o.squeeze(2)).abs() <= 5.3 * 2 ** -7)
                assert torch.all((lse1 - lse.squeeze(2)).abs() <= 1e-3)
            out.append((o, lse))
            lens = new
        return pool, torch.cat([o for o, _ in out], 2), torch.cat([l for _, l in out], 2)

    pool, o, lse = run([0, T + 1])
    pool2, o2, lse2 = run([0, 77, T, T + 1])
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert torch.equal(pool, pool2)
    # rows of a chunk see the same tiles in the same order
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
