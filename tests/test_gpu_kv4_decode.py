"""paged_kv4_attn_decode against the fp64 oracle over the values the 4-bit cache holds
(every one of them is a bf16, so the oracle's bf16 pools hold them exactly).

Tolerances.  O: the result is rounded to bf16 (2^-8 of |O|) and each product p t before
(2^-8 of sum p |v|); fp32 accumulation of at most 2^5 steps of 4 products adds less than
2^-16 of sum p |v|.  LSE: a group's score starts from -8 sum q and adds 32 products of at
most 15 |q|, in four adds of 8 products, each good to 2^-22 of 23 sum |q|; so 2^-20 of that,
times the largest scale of the group, summed over groups, times the softmax scale; plus
2^-20 of |LSE| and 2^-18 for exponentials, sums and logarithms.
"""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import rope_ref as ref
import synth
from gpu_util import from_dev, to_dev, to_dev_i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


class Cache:
    """A paged batch in both forms: the 4-bit pool and the bf16 pools of its values."""

    def __init__(self, lens, Hq, Hkv, D, seed, gain=1.0, max_len=None):
        cfg = synth.DecodeConfig("kv4", len(lens), Hq, Hkv, D, 0, 1, 16, seed, mult=gain)
        p = synth.paged_inputs(cfg, seq_lens=lens, max_seq_len=max_len or max(max(lens), 1))
        p.q = synth.normal_bf16(seed + 9, p.q.shape)
        self.p, self.scale = p, cfg.softmax_scale
        # dead slots hold NaN in the bf16 pools, so they hold NaN scales here
        self.pool_host = ref.pool_from_bf16(p.k_pool, p.v_pool)
        self.k, self.v = ref.value_bits(p.k_pool), ref.value_bits(p.v_pool)
        self.pool = torch.from_numpy(self.pool_host).cuda()
        self.table, self.lens = to_dev_i32(p.block_table), to_dev_i32(p.seq_lens)
        self.q = to_dev(p.q)

    def expect(self):
        p = self.p
        o, lse = oracle.paged_decode(p.q, self.k, self.v, p.block_table, p.seq_lens, self.scale)
        a, _ = oracle.paged_decode(p.q, self.k, self.v & 0x7FFF, p.block_table, p.seq_lens, self.scale)
        return o, lse, (2.0 ** -8 + 2.0 ** -16) * a

    def lse_tolerance(self, lse):
        p = self.p
        S, Hq, D = p.q.shape
        Hkv = p.k_pool.shape[1]
        scales = synth.bf16_bits_to_float(ref.quantise(p.k_pool)[1]).astype(np.float64)
        big = np.nanmax(np.where(np.isnan(scales), 0, scales), (0, 2))  # [Hkv, groups]
        q = np.abs(synth.bf16_bits_to_float(p.q).astype(np.float64)).reshape(S, Hq, -1, 32).sum(-1)
        s = (q * np.repeat(big, Hq // Hkv, 0)).sum(-1)
        fin = np.where(np.isfinite(lse), np.abs(lse), 0)
        return 2.0 ** -20 * 23 * self.scale * s + 2.0 ** -20 * fin + 2.0 ** -18


def check(c, o, lse, rows=None):
    want, wl, more = c.expect()
    got, gl = from_dev(o), from_dev(lse)
    tol = 2.0 ** -8 * np.abs(want) + more
    ltol = c.lse_tolerance(wl)
    rows = range(len(want)) if rows is None else rows
    for r in rows:
        if c.p.seq_lens[r] == 0:
            assert np.all(got[r] == 0) and np.all(np.isneginf(gl[r]))
            continue
        assert np.all(np.abs(got[r] - want[r]) <= tol[r]), (r, np.max(np.abs(got[r] - want[r]) - tol[r]))
        assert np.all(np.abs(gl[r] - wl[r]) <= ltol[r]), (r, np.max(np.abs(gl[r] - wl[r]) - ltol[r]))


CASES = [
    ([1], 1, 1, 128),
    ([16, 17, 64, 65, 63], 4, 2, 128),
    ([1, 0, 15, 300, 0, 33], 8, 1, 64),
    ([5, 129, 1000, 256, 257], 16, 1, 64),     # 16 query heads on one KV head
    ([700, 1, 48], 12, 1, 128),
    ([4000, 513, 2], 6, 3, 128),
    ([2047, 31], 5, 5, 64),
    ([40], 16, 1, 128),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D", CASES)
def test_decode_matches_the_oracle(gb, lens, Hq, Hkv, D):
    c = Cache(lens, Hq, Hkv, D, 50000 + sum(lens))
    # up to 1024 tokens one launch without a workspace, above that the split and its merge
    for bound in {c.p.max_seq_len, max(c.p.max_seq_len, 1025)}:
        need = gb.paged_kv4_attn_decode_workspace_size(len(lens), Hq, Hkv, D, bound)
        assert (need == 0) == (bound <= 1024)
        o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, bound, scale=c.scale)
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_OK, 0)
        check(c, o, lse)


@pytest.mark.parametrize("gain", [0.01, 30.0])
def test_small_and_large_cache_values(gb, gain):
    c = Cache([100, 777], 8, 2, 128, 51000, gain)
    o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, c.p.max_seq_len, scale=c.scale)
    check(c, o, lse)


def shifted(bits, k):
    """bf16 bits times 2^k; zeros and NaN stay."""
    e = (bits >> 7) & 0xFF
    move = (e > 0) & (e < 0xFF)
    assert not move.any() or 0 < int(e[move].min()) + k and int(e[move].max()) + k < 0xFF
    return np.where(move, bits + np.uint16(k * 128 % 65536), bits).astype(np.uint16)


def shift_keys(pool, D, k):
    """A 4-bit pool whose keys are times 2^k (their scales are)."""
    out = pool.copy()
    scales = np.ascontiguousarray(out[..., 8 * D:9 * D]).view(np.uint16)
    out[..., 8 * D:9 * D] = np.ascontiguousarray(shifted(scales, k)).view(np.uint8)
    return out


@pytest.mark.parametrize("k", [-104, 60, 95, 101, 107, 113, 118])
@pytest.mark.parametrize("Hq,Hkv,D", [(6, 2, 128), (12, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("bound", [700, 1100])
def test_queries_of_any_magnitude(gb, Hq, Hkv, D, k, bound):
    """Queries times 2^k on keys times 2^-k: the same scores, however large the queries.
    (What fp32 sums below 2^-126 lose, 2^-150 of a key of 2^-118 against a query of 2^118,
    is 2^-18 of a score, within the tolerances' 2^-16.)"""
    c = Cache([700, 1, 90], Hq, Hkv, D, 51500 + Hq, max_len=bound)
    bits = c.p.q.copy()
    bits[((bits >> 7) & 0xFF) < 127 - 12] = 0  # (so that every element of the row can be shifted)
    bits[1, 0] = 0                             # a row of zeros
    c.p.q = bits
    q, pool = to_dev(shifted(bits, k)), torch.from_numpy(shift_keys(c.pool_host, D, -k)).cuda()
    o, lse = gb.paged_kv4_attn_decode(q, pool, c.table, c.lens, bound, scale=c.scale)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    check(c, o, lse)
    if k in (-104, 60, 95):  # (products and sums of 2^k times the fp32 values, none subnormal)
        o1, lse1 = gb.paged_kv4_attn_decode(to_dev(bits), c.pool, c.table, c.lens, bound, scale=c.scale)
        assert torch.equal(o, o1) and torch.equal(lse, lse1)


@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e-12])
@pytest.mark.parametrize("bound", [300, 1100])
def test_tiny_softmax_scales(gb, scale, bound):
    """Scores of nothing: the mean of the values, also of rows of zeros."""
    c = Cache([300, 64, 1], 4, 2, 128, 51700, max_len=bound)
    c.p.q[0] = 0
    c.q, c.scale = to_dev(c.p.q), scale
    o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, bound, scale=scale)
    check(c, o, lse)


def test_the_largest_length_bound(gb):
    """Any bound an int holds."""
    c = Cache([700, 1, 90], 6, 2, 128, 51800, max_len=1100)
    o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, 2 ** 31 - 1, scale=c.scale)
    check(c, o, lse)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)


def test_the_decode_workload(gb):
    cfg = synth.CONFIGS["paged_decode"]
    lens = synth.uniform_ints(cfg.seed + 3, cfg.num_seqs, cfg.len_lo, cfg.len_hi)
    c = Cache(list(lens), cfg.Hq, cfg.Hkv, cfg.D, cfg.seed)
    o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, c.p.max_seq_len, scale=c.scale)
    check(c, o, lse)
    # the same bits wherever the blocks sit, on another stream, and without an LSE
    perm = synth.permutation(77, c.p.num_pool_blocks)
    pool2 = torch.empty_like(c.pool)
    pool2[torch.from_numpy(perm).cuda()] = c.pool
    t2 = to_dev_i32(np.where(c.p.block_table >= 0, perm[c.p.block_table], -1))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, none = gb.paged_kv4_attn_decode(c.q, pool2, t2, c.lens, c.p.max_seq_len, scale=c.scale,
                                        return_lse=False, stream=s)
    s.synchronize()
    assert none is None and torch.equal(o, o2)


def test_many_short_requests(gb):
    lens = list(synth.uniform_ints(52000, 300, 0, 40))
    c = Cache(lens, 4, 2, 64, 52001, max_len=512)
    for bound in (512, 2000):
        o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, bound, scale=c.scale)
        check(c, o, lse)


def test_one_long_request_at_large_offsets(gb):
    """A pool past 2^31 bytes with the request's blocks at its far end."""
    L, Hkv, D = 20000, 2, 128
    c = Cache([L], 8, Hkv, D, 53000)
    extra = (1 << 31) // (Hkv * 18 * D) + 10
    pool = torch.empty((extra + c.pool.shape[0], Hkv, 18 * D), dtype=torch.uint8, device="cuda")
    pool[extra:] = c.pool
    table = torch.where(c.table >= 0, c.table + extra, -1).int()
    o, lse = gb.paged_kv4_attn_decode(c.q, pool, table, c.lens, L, scale=c.scale)
    check(c, o, lse)
    k, _ = gb.paged_kv4_gather(pool, table, c.lens, L)
    k0, _ = gb.paged_kv4_gather(c.pool, c.table, c.lens, L)
    assert torch.equal(k, k0)


@pytest.mark.parametrize("bound", [70, 1100])
def test_nan_in_the_cache_stays_where_it_is_read(gb, bound):
    lens = [50, 60, 70]
    c = Cache(lens, 4, 2, 128, 54000)
    host = c.pool_host.copy()
    D = 128
    blk = c.p.block_table
    host[blk[1, 2], 0, 8 * D + 3 * 8:8 * D + 3 * 8 + 2] = [0xC0, 0x7F]       # K, head 0, group 0
    host[blk[2, 1], 1, 17 * D + 5 * 8 + 2:17 * D + 5 * 8 + 4] = [0xC0, 0x7F]  # V, head 1, group 1
    o, lse = gb.paged_kv4_attn_decode(c.q, torch.from_numpy(host).cuda(), c.table, c.lens, bound,
                                      scale=c.scale)
    check(c, o, lse, rows=[0])
    nan = from_dev(o) != from_dev(o)
    assert nan[1, :2].all() and not nan[1, 2:].any()
    assert nan[2, 2:, 32:64].all() and not nan[2, :2].any()
    assert not nan[2, 2:, :32].any() and not nan[2, 2:, 64:].any()
    ln = torch.isnan(lse).cpu().tolist()
    assert ln == [[False] * 4, [True, True, False, False], [False] * 4]


@pytest.mark.parametrize("bound", [400, 1100])
def test_bad_requests_are_flagged(gb, bound):
    c = Cache([100, 200, 300, 400], 4, 2, 64, 55000)
    table = c.p.block_table.copy()
    table[1, 5] = c.p.num_pool_blocks
    table[1, 12] = -3
    lens = c.p.seq_lens.copy()
    lens[2] = bound + 1
    lens[3] = -1
    o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, to_dev_i32(table), to_dev_i32(lens), bound,
                                      scale=c.scale)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2 | 4)
    assert torch.isnan(o[1:]).all() and torch.isnan(lse[1:]).all()
    check(c, o, lse, rows=[0])


@pytest.mark.parametrize("bound", [200, 1100])
def test_a_wait_that_runs_out_is_reported(gb, bound):
    c = Cache([100, 200], 4, 2, 64, 56000)
    gb.test_set_failure(2_000_000, True)
    try:
        gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, bound, scale=c.scale)
        torch.cuda.synchronize()
        st, flags = gb.attn_device_status()
    finally:
        gb.test_set_failure(0, False)
    assert st == gb.ATTN_ERR_DEVICE and flags & 1
    o, lse = gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, bound, scale=c.scale)
    check(c, o, lse)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)


def test_decode_steps_from_projections_replayed_as_a_graph(gb):
    """A model's step -- norm, rotation, quantised append, attention -- captured once and
    replayed, against the same calls made one by one, and against the oracle at the end."""
    lens, Hq, Hkv, D, steps = [0, 15, 16, 200, 1023], 12, 2, 128, 20
    S = len(lens)
    room = max(lens) + steps
    bt = np.arange(S * (room // 16 + 1), dtype=np.int32).reshape(S, -1)[:, ::-1].copy()
    cs = torch.from_numpy(ref.table(room, D)).cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    kb, vb = synth.normal_bf16(57000, (2, bt.size, Hkv, 16, D))
    rows = [to_dev(synth.normal_bf16(57100 + i, (S, 1, Hq + 2 * Hkv, D))) for i in range(steps)]

    class State:
        def __init__(self):
            self.pool = torch.from_numpy(ref.pool_from_bf16(kb, vb)).cuda()
            self.table, self.lens = to_dev_i32(bt), to_dev_i32(np.array(lens))
            self.new = torch.empty_like(self.lens)
            self.rows = torch.empty_like(rows[0])
            self.qr = torch.empty((S, Hq, 1, D), dtype=torch.bfloat16, device="cuda")
            self.o = torch.empty((S, Hq, D), dtype=torch.bfloat16, device="cuda")
            self.lse = torch.empty((S, Hq), dtype=torch.float32, device="cuda")
            n = gb.paged_kv4_attn_decode_workspace_size(S, Hq, Hkv, D, room)
            self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

        def step(self):
            q, k, v = self.rows.split([Hq, Hkv, Hkv], 2)
            gb.paged_kv4_append(q, k, v, self.pool, self.table, self.lens, cs, w, w, q_out=self.qr,
                                new_seq_lens=self.new)
            gb.paged_kv4_attn_decode(self.qr.view(S, Hq, D), self.pool, self.table, self.new, room,
                                     out=self.o, lse=self.lse, workspace=self.ws)
            self.lens.copy_(self.new)

    warm, eager, graphed = State(), State(), State()
    warm.rows.copy_(rows[0])
    warm.step()
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        graphed.step()
    for x in rows:
        eager.rows.copy_(x)
        eager.step()
        graphed.rows.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.o, graphed.o) and torch.equal(eager.lse, graphed.lse)
    assert torch.equal(eager.pool, graphed.pool)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    kg, vg = gb.paged_kv4_gather(eager.pool, eager.table, eager.lens, room)
    for r, n in enumerate(lens):
        kf, vf = (from_dev(t[r, :, :n + steps]) for t in (kg, vg))
        q = from_dev(eager.qr)[r, :, 0].reshape(Hkv, -1, D)
        s = np.einsum("hgd,htd->hgt", q, kf) / np.sqrt(D)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want = np.einsum("hgt,htd->hgd", p, vf).reshape(Hq, D)
        mag = np.einsum("hgt,htd->hgd", p, np.abs(vf)).reshape(Hq, D)
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -16) * mag
        assert np.all(np.abs(from_dev(eager.o)[r] - want) <= tol)


def test_both_bindings_give_the_same_bits(gb, monkeypatch):
    """The compiled way into the library and the Python code behind it, with what may be
    given and what may be left out; refused calls name the fault either way."""
    gb._load_torch()
    assert gb._quick is not None
    S, Hq, Hkv, D, L = 4, 8, 2, 128, 1500
    c = Cache([1, 700, 1500, 33], Hq, Hkv, D, 58000)
    q4 = to_dev(synth.normal_bf16(58100, (S, Hq, 3, D)))
    out, lse = torch.empty_like(c.q), torch.empty((S, Hq), device="cuda")
    ws = torch.empty(gb.paged_kv4_attn_decode_workspace_size(S, Hq, Hkv, D, L), dtype=torch.uint8,
                     device="cuda")
    cache = (c.pool, c.table, c.lens, L)

    def calls():
        yield gb.paged_kv4_attn_decode(c.q, *cache)
        yield gb.paged_kv4_attn_decode(c.q, *cache, scale=0.2, return_lse=False)
        yield gb.paged_kv4_attn_decode(c.q, *cache, scale=1, out=out, lse=lse, workspace=ws)
        yield gb.paged_kv4_attn_prefill(q4, *cache, causal=True)
        yield gb.paged_kv4_attn_prefill(q4, *cache, causal=False, return_lse=False)
        yield gb.paged_kv4_gather(*cache)
        yield gb.paged_kv4_gather(*cache, k_out=torch.zeros((S, Hkv, L, D), dtype=torch.bfloat16,
                                                            device="cuda"),
                                  v_out=torch.zeros((S, Hkv, L, D), dtype=torch.bfloat16,
                                                    device="cuda"))

    def results():
        return [tuple(None if t is None else t.clone() for t in r) for r in calls()]

    quick = results()
    with pytest.raises(ValueError):
        gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens[:2], L)
    with pytest.raises(ValueError):
        gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, L, workspace=ws.float())
    with pytest.raises(gb.GbAttnError):
        gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, L, workspace=ws[:256])
    with pytest.raises(gb.GbAttnError):
        gb.paged_kv4_attn_decode(c.q, c.pool, c.table, c.lens, L, scale=float("nan"))
    with pytest.raises(TypeError):
        gb.paged_kv4_attn_decode([1], c.pool, c.table, c.lens, L)
    monkeypatch.setattr(gb, "_quick", None)
    for a, b in zip(quick, results()):
        assert len(a) == len(b)
        for x, y in zip(a, b):
            assert (x is None) == (y is None)
            # (values past the end are left as they were: NaN keeps its bits)
            assert x is None or torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                                            y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32))
