"""paged_kv4_attn_prefill: its tile kernel against the bf16 paged prefill over the same
values (equal bits: every value the 4-bit cache holds is a bf16), its row kernels (short
chunks) against the fp64 oracle, with the tolerances of the 4-bit decode, and both on the
inputs where they could go wrong."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import rope_ref as ref
import synth
from gpu_util import check_close, from_dev, to_dev, to_dev_i32
from test_gpu_kv4_decode import shift_keys, shifted

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


class Item:
    def __init__(self, Hq, Hkv, D, Tq, lens, seed, max_len=0):
        cfg = synth.DecodeConfig("kv4p", len(lens), Hq, Hkv, D, 0, 1, 16, seed)
        p = synth.paged_inputs(cfg, seq_lens=lens, max_seq_len=max(max(lens), 1, max_len))
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


def uses_rows(gb, c):
    B, Hq, Tq, D = c.q.shape
    return gb.paged_kv4_attn_prefill_workspace_size(B, Hq, c.p.k_pool.shape[1], Tq, D,
                                                    c.p.max_seq_len) > 0


TILES = [
    # Hq, Hkv, D, Tq, kv_lens
    (8, 2, 128, 512, [512, 700, 5000, 8192]),
    (12, 2, 128, 300, [300, 301, 1024, 2999]),
    (4, 4, 64, 257, [257, 640, 1000, 4096]),
    (16, 2, 64, 512, [600, 8192]),
    (32, 4, 128, 64, [64, 100, 2049, 4000, 129, 128]),
    (32, 2, 128, 70, [0, 5, 69, 70, 128, 129]),   # chunks longer than their cache
    (24, 1, 64, 130, [0, 1, 15, 16, 17, 127]),
]

ROWS = [
    (8, 2, 128, 1, [1, 17, 4096, 8192]),
    (8, 2, 128, 4, [4, 5, 63, 64, 65, 300]),      # 16 rows on a KV head
    (3, 1, 128, 3, [3, 70, 700]),                 # 9 rows
    (5, 5, 64, 7, [7, 8, 1000]),                  # 7 rows, no sharing
    (8, 2, 64, 5, [100, 0, 3, 4, 5, 129]),        # 20 rows: two chunks, caches below Tq
    (32, 2, 128, 6, [6, 900]),                    # 96 rows
    (2, 1, 128, 37, [0, 5, 36, 37, 128, 129]),
    (2, 1, 64, 130, [0, 1, 15, 16, 17, 127]),
    (4, 2, 128, 200, [200, 333]),
]


@pytest.mark.parametrize("Hq,Hkv,D,Tq,lens", TILES)
@pytest.mark.parametrize("causal", [True, False])
def test_tiles_equal_the_bf16_prefill_over_the_same_values(gb, Hq, Hkv, D, Tq, lens, causal):
    c = Item(Hq, Hkv, D, Tq, lens, 60000 + Tq)
    assert not uses_rows(gb, c)
    o, lse = c.run(gb, causal)
    o2, lse2 = gb.paged_attn_prefill(c.q, to_dev(c.k), to_dev(c.v), c.table, c.kv_lens,
                                     c.p.max_seq_len, causal=causal, scale=c.scale)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,Hkv,D,Tq,lens", [TILES[1], TILES[2], TILES[5], TILES[6]])
def test_tiles_match_the_oracle(gb, Hq, Hkv, D, Tq, lens):
    c = Item(Hq, Hkv, D, Tq, lens, 61000 + Tq)
    o, lse = c.run(gb, True)
    o_ref, l_ref = oracle.paged_prefill(c.q_bits, c.k, c.v, c.p.block_table, c.p.seq_lens, True,
                                        c.scale)
    og, lg = from_dev(o), from_dev(lse)
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lg), empty) and np.all(og[empty] == 0)
    check_close(og[~empty], lg[~empty], o_ref[~empty], l_ref[~empty], "kv4 prefill")


def check_rows(c, o, lse, causal, items=None):
    """Tolerances as derived in test_gpu_kv4_decode.py."""
    p = c.p
    args = (p.block_table, p.seq_lens, causal, c.scale)
    want, wl = oracle.paged_prefill(c.q_bits, c.k, c.v, *args)
    mag, _ = oracle.paged_prefill(c.q_bits, c.k, c.v & 0x7FFF, *args)
    B, Hq, Tq, D = c.q_bits.shape
    Hkv = p.k_pool.shape[1]
    scales = synth.bf16_bits_to_float(ref.quantise(p.k_pool)[1]).astype(np.float64)
    big = np.nanmax(np.where(np.isnan(scales), 0, scales), (0, 2))  # [Hkv, groups]
    qs = np.abs(synth.bf16_bits_to_float(c.q_bits).astype(np.float64))
    qs = qs.reshape(B, Hq, Tq, -1, 32).sum(-1)
    s = (qs * np.repeat(big, Hq // Hkv, 0)[None, :, None]).sum(-1)
    fin = np.where(np.isfinite(wl), np.abs(wl), 0)
    ltol = 2.0 ** -20 * 23 * c.scale * s + 2.0 ** -20 * fin + 2.0 ** -18
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -16) * mag
    got, gl = from_dev(o), from_dev(lse)
    empty = np.isneginf(wl)
    for b in range(B) if items is None else items:
        e = empty[b]
        assert np.array_equal(np.isneginf(gl[b]), e) and np.all(got[b][e] == 0), b
        assert np.all(np.abs(got[b] - want[b])[~e] <= tol[b][~e]), b
        assert np.all(np.abs(gl[b][~e] - wl[b][~e]) <= ltol[b][~e]), b


@pytest.mark.parametrize("Hq,Hkv,D,Tq,lens", ROWS)
@pytest.mark.parametrize("causal", [True, False])
def test_rows_match_the_oracle(gb, Hq, Hkv, D, Tq, lens, causal):
    c = Item(Hq, Hkv, D, Tq, lens, 60500 + Tq, max_len=1000)
    assert uses_rows(gb, c)
    o, lse = c.run(gb, causal)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    check_rows(c, o, lse, causal)


@pytest.mark.parametrize("k", [60, 101, 118])
@pytest.mark.parametrize("Hq,Hkv,D,Tq", [(8, 2, 128, 4), (4, 2, 64, 2), (32, 1, 128, 1)])
def test_row_queries_of_any_magnitude(gb, Hq, Hkv, D, Tq, k):
    """Queries times 2^k on keys times 2^-k, as in test_gpu_kv4_decode.py."""
    c = Item(Hq, Hkv, D, Tq, [Tq, 65, 700], 61300 + Tq, max_len=1000)
    assert uses_rows(gb, c)
    c.q_bits[((c.q_bits >> 7) & 0xFF) < 127 - 12] = 0
    c.q = to_dev(shifted(c.q_bits, k))
    o, lse = c.run(gb, True, pool=torch.from_numpy(shift_keys(c.pool_host, D, -k)).cuda())
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    check_rows(c, o, lse, True)


@pytest.mark.parametrize("Hq,Hkv,D", [(17, 1, 128), (24, 1, 64), (32, 1, 128), (34, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("max_len", [512, 513, 1024, 1025])
def test_one_token_of_wide_groups(gb, Hq, Hkv, D, max_len):
    """Single tokens of more than 16 query heads on a KV head, on both sides of every length
    bound at which the kernels change; what lies around the outputs stays as it was."""
    c = Item(Hq, Hkv, D, 1, [1, 0, 17, 64, 65, 300, 500, 512, 511], 61400 + Hq + max_len, max_len=max_len)
    B = len(c.lens)
    # (16 heads are one pass: a single launch without a workspace up to 1024 keys)
    wide = Hq // Hkv > 16
    assert uses_rows(gb, c) == ((max_len > 512 or B * Hq > 152) if wide else max_len > 1024)
    n = B * Hq
    for causal in (True, False):
        around = torch.full((3 * n * D,), 7.0, dtype=torch.bfloat16, device="cuda")
        around_lse = torch.full((3 * n,), 7.0, device="cuda")
        o = around[n * D:2 * n * D].view(B, Hq, 1, D)
        lse = around_lse[n:2 * n].view(B, Hq, 1)
        c.run(gb, causal, out=o, lse=lse)
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_OK, 0)
        check_rows(c, o, lse, causal)
        assert torch.all(around[:n * D] == 7) and torch.all(around[2 * n * D:] == 7)
        assert torch.all(around_lse[:n] == 7) and torch.all(around_lse[2 * n:] == 7)


def test_one_drafted_token_equals_the_decode(gb):
    c = Item(12, 2, 128, 1, [1, 300, 4000], 61500)  # (past the decode's one-launch form)
    o, lse = c.run(gb, True)
    o2, lse2 = gb.paged_kv4_attn_decode(c.q.squeeze(2), c.pool, c.table, c.kv_lens, 4000,
                                        scale=c.scale)
    assert torch.equal(o.squeeze(2), o2) and torch.equal(lse.squeeze(2), lse2)


def test_more_classes_than_the_sorted_list_holds(gb):
    """More (item, query pair) classes than are sorted: the items' own order."""
    lens = list(synth.uniform_ints(61600, 400, 0, 90))
    c = Item(2, 1, 64, 40, lens, 61601)
    assert not uses_rows(gb, c)
    o, lse = c.run(gb, True)
    o2, lse2 = gb.paged_attn_prefill(c.q, to_dev(c.k), to_dev(c.v), c.table, c.kv_lens,
                                     c.p.max_seq_len, causal=True, scale=c.scale)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_length_bound_of_any_size(gb):
    """Short chunks under the largest bound an int holds: more steps than the row kernels
    count, so tiles."""
    c = Item(4, 2, 128, 4, [4, 70, 333, 0] * 8, 61700)
    top = 2 ** 31 - 1
    o, lse = gb.paged_kv4_attn_prefill(c.q, c.pool, c.table, c.kv_lens, top, scale=c.scale)
    o2, lse2 = gb.paged_attn_prefill(c.q, to_dev(c.k), to_dev(c.v), c.table, c.kv_lens, top,
                                     scale=c.scale)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


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


PATHS = [(20, 1000), (20, 0), (300, 0)]  # Tq, max_len: by rows, by tiles, by tiles


@pytest.mark.parametrize("Tq,max_len", PATHS)
def test_nan_keys_reach_the_queries_that_see_them(gb, Tq, max_len):
    D = 128
    c = Item(4, 2, D, Tq, [Tq + 20] * 2, 63000, max_len)
    assert uses_rows(gb, c) == (max_len > 0)
    host = c.pool_host.copy()
    blk = c.p.block_table
    # token 30 of item 0: its key in head 0 (seen by queries 10 and on)
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


@pytest.mark.parametrize("Tq,max_len", PATHS)
def test_bad_requests_are_flagged(gb, Tq, max_len):
    c = Item(4, 2, 64, Tq, [100, 200, 300, 100], 64000, max_len)
    table = c.p.block_table.copy()
    table[1, 5] = c.p.num_pool_blocks
    lens = c.p.seq_lens.copy()
    lens[2], lens[3] = c.p.max_seq_len + 1, -1
    o, lse = c.run(gb, True, table=to_dev_i32(table), lens=to_dev_i32(lens))
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2 | 4)
    assert torch.isnan(o[2:]).all() and torch.isnan(lse[2:]).all()
    good, _ = c.run(gb, True)
    assert torch.equal(o[0], good[0])  # item 1 read another block: unspecified
    if uses_rows(gb, c):
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("Tq,max_len", PATHS)
def test_a_wait_that_runs_out_is_reported(gb, Tq, max_len):
    c = Item(4, 2, 128, Tq, [100, 200], 65000, max_len)
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
    """A prompt through the whole path in chunks -- projection rows, norm, rotation,
    quantised append, attention -- against the prompt in one chunk."""
    Hq, Hkv, D, T = 8, 2, 128, 320
    rows = to_dev(synth.normal_bf16(66000, (2, T + 1, Hq + 2 * Hkv, D)))
    cs = torch.from_numpy(ref.table(T + 1, D)).cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    table = to_dev_i32(np.pad(synth.permutation(9, 44).reshape(2, 22), ((0, 0), (0, 48))))
    v_max = float(rows[:, :, Hq + Hkv:].abs().max())

    def run(cuts):
        pool = torch.zeros((44, Hkv, 18 * D), dtype=torch.uint8, device="cuda")
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        out = []
        for a, b in zip(cuts, cuts[1:]):
            q, k, v = rows[:, a:b].split([Hq, Hkv, Hkv], 2)
            new = torch.empty_like(lens)
            q, _ = gb.paged_kv4_append(q, k, v, pool, table, lens, cs, w, w, new_seq_lens=new)
            out.append(gb.paged_kv4_attn_prefill(q, pool, table, new, 1000))
            lens = new
        return pool, torch.cat([o for o, _ in out], 2), torch.cat([l for _, l in out], 2)

    pool, o, lse = run([0, T + 1])                 # tiles
    pool2, o2, lse2 = run([0, 270, T - 3, T, T + 1])  # tiles, rows, rows, one row
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert torch.equal(pool, pool2)
    # tile rows see the same tiles in the same order
    assert torch.equal(o[:, :, :270], o2[:, :, :270]) and torch.equal(lse[:, :, :270], lse2[:, :, :270])
    # the kernels round probabilities and results at different points: 2^-8 of sum p |v| and
    # of |O| each, twice; values are at most v_max (1 + 2^-5) in the cache
    assert torch.all((o - o2).abs() <= 4 * 2.0 ** -8 * v_max * (1 + 2.0 ** -5))
    assert torch.all((lse - lse2).abs() <= 1e-4)


def test_calls_in_a_row_equal_calls_apart(gb):
    """The kernels let their successors be set up before they end.  A chain of calls in the
    same buffers, each reading or overwriting what the one before wrote, gives the bits of
    the same chain with a synchronisation after every call."""
    S, Hq, Hkv, D, Tn, rounds, first = 16, 8, 2, 128, 64, 6, 1500
    room = first + 16 * S + rounds * (Tn + 1)
    bt = np.random.default_rng(9).permutation(S * (room // 16 + 1)).reshape(S, -1).astype(np.int32)
    kb, vb = synth.normal_bf16(59000, (2, bt.size, Hkv, 16, D))
    start = first + 16 * np.arange(S)
    lens = [to_dev_i32(start + i * (Tn + 1)) for i in range(rounds)]
    more = [to_dev_i32(start + i * (Tn + 1) + Tn) for i in range(rounds)]
    last = [to_dev_i32(start + i * (Tn + 1) + Tn + 1) for i in range(rounds)]
    rows = [to_dev(synth.normal_bf16(59100 + i, (S, Tn, Hq + 2 * Hkv, D))) for i in range(rounds)]
    cs = torch.from_numpy(ref.table(room, D)).cuda()
    w = to_dev(synth.float_to_bf16_bits((1 + 0.2 * synth.normals(59200, D)).astype(np.float32)))
    how = dict(cos_sin=cs, q_weight=w, k_weight=w)

    def chain(wait):
        dev = dict(device="cuda")
        pool = torch.from_numpy(ref.pool_from_bf16(kb, vb)).cuda()
        table = to_dev_i32(bt)
        new = torch.empty(S, dtype=torch.int32, **dev)
        qkv = [torch.empty((S, h, Tn, D), dtype=torch.bfloat16, **dev) for h in (Hq, Hkv, Hkv)]
        d = [torch.empty((S, Tn, h, D), dtype=torch.bfloat16, **dev) for h in (Hq, Hkv, Hkv)]
        dw = torch.empty((2, D), **dev)
        wsb = torch.empty(gb.qkv_norm_rope_bwd_workspace_size(S, Tn, D), dtype=torch.uint8, **dev)
        ws = torch.empty(gb.paged_kv4_attn_decode_workspace_size(S, Hq, Hkv, D, room),
                         dtype=torch.uint8, **dev)
        assert ws.numel() > 0 and gb.paged_kv4_attn_prefill_workspace_size(S, Hq, Hkv, Tn, D, room) == 0
        q1 = torch.empty((S, Hq, 1, D), dtype=torch.bfloat16, **dev)
        hist = [torch.zeros((S, Hkv, room, D), dtype=torch.bfloat16, **dev) for _ in range(2)]
        o, lse = torch.empty_like(qkv[0]), torch.empty((S, Hq, Tn), **dev)
        o1, lse1 = torch.empty((S, Hq, D), dtype=torch.bfloat16, **dev), torch.empty((S, Hq), **dev)
        out = []
        for i in range(rounds):
            q, k, v = rows[i].split([Hq, Hkv, Hkv], 2)
            calls = [
                lambda: gb.qkv_norm_rope(q, k, v, q_out=qkv[0], k_out=qkv[1], v_out=qkv[2], **how),
                lambda: gb.qkv_norm_rope_bwd(*qkv, q, k, dq=d[0], dk=d[1], dv=d[2], dq_weight=dw[0],
                                             dk_weight=dw[1], workspace=wsb, **how),
                lambda: gb.paged_kv4_append(d[0], d[1], d[2], pool, table, lens[i], q_out=qkv[0],
                                            new_seq_lens=new, **how),
                lambda: gb.paged_kv4_gather(pool, table, new, room, k_out=hist[0], v_out=hist[1]),
                lambda: gb.paged_kv4_attn_prefill(qkv[0], pool, table, more[i], room, out=o, lse=lse),
                lambda: gb.paged_kv4_append(q[:, :1], k[:, :1], v[:, :1], pool, table, new, q_out=q1,
                                            **how),
                lambda: gb.paged_kv4_attn_decode(q1[:, :, 0], pool, table, last[i], room, out=o1,
                                                 lse=lse1, workspace=ws),
                lambda: gb.paged_kv4_append(None, k[:, :1], v[:, :1], pool, table, new, **how),
                lambda: gb.paged_kv4_attn_decode(q1[:, :, 0], pool, table, last[i], room, out=o1,
                                                 lse=lse1, workspace=ws),
            ]
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
            out += [t.clone() for t in (*qkv, *d, dw, pool, *hist, o, lse, o1, lse1)]
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_OK, 0)
        return out

    apart = chain(True)
    for _ in range(3):
        for a, b in zip(apart, chain(False)):
            assert torch.equal(a, b)
    assert all(t.isfinite().all() for t in apart if t.is_floating_point())
