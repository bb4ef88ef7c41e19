"""paged_kv_keep moves the kept rows bit for bit and touches nothing else, and a whole step
with drafted tokens: append, tree attention, verification, keeping."""

from __future__ import annotations

import numpy as np
import pytest

import synth
import tree_ref as ref
from gpu_util import bits_of, from_dev, to_dev, to_dev_i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


class Cache:
    """Pools of any bits, a table, and paths of kept rows."""

    def __init__(self, S, Hkv, D, n, lens, layers, seed, counts=None, dense=False):
        rng = np.random.default_rng(seed)
        self.lens = np.array(lens, dtype=np.int32)
        self.counts = np.array(counts if counts is not None else rng.integers(0, n + 1, S))
        self.path = np.full((S, n), -1)
        for r, c in enumerate(self.counts):
            span = c if dense else 2 * n
            self.path[r, :c] = np.sort(rng.choice(max(span, c), c, replace=False))
        blocks = -(-(self.lens + 2 * n) // 16)
        NB = int(blocks.sum()) + 3
        perm = rng.permutation(NB)
        self.table = np.full((S, int(blocks.max()) + 1), -1)
        at = 0
        for r, b in enumerate(blocks):
            self.table[r, :b] = perm[at:at + b]
            at += b
        self.pools = rng.integers(0, 1 << 16, (2, layers, NB, Hkv, 16, D)).astype(np.uint16)

    def dev(self):
        pools = torch.from_numpy(self.pools.view(np.int16)).view(torch.bfloat16).cuda()
        return pools, [to_dev_i32(x) for x in (self.table, self.lens, self.path, self.counts)]

    def want(self):
        return np.stack([np.stack([ref.keep(l, self.table, self.lens, self.path, self.counts)
                                   for l in kv]) for kv in self.pools])


CASES = [
    # S, Hkv, D, path entries, lens, layers
    (5, 2, 128, 8, [0, 1, 15, 16, 100], 1),
    (5, 2, 64, 8, [0, 1, 15, 16, 100], 3),
    (3, 1, 64, 1, [7, 0, 31], 2),
    (4, 3, 128, 40, [0, 9, 200, 33], 5),
    (2, 8, 128, 256, [3, 500], 2),
    (1, 1, 128, 17, [15], 40),
    (200, 2, 64, 6, list(range(200)), 2),
]


@pytest.mark.parametrize("S,Hkv,D,n,lens,layers", CASES)
def test_rows_move_bit_for_bit(gb, S, Hkv, D, n, lens, layers):
    c = Cache(S, Hkv, D, n, lens, layers, 90000 + n)
    pools, args = c.dev()
    new = torch.full((S + 2,), 77, dtype=torch.int32, device="cuda")
    got = gb.paged_kv_keep(pools[0], pools[1], *args, new_seq_lens=new[1:-1])
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert np.array_equal(bits_of(pools), c.want())
    assert got.tolist() == (c.lens + c.counts).tolist() and new[0] == 77 and new[-1] == 77
    # a sequence of pools, no lengths asked for
    pools, args = c.dev()
    assert gb.paged_kv_keep(list(pools[0]), tuple(pools[1]), *args) is None
    assert np.array_equal(bits_of(pools), c.want())


def test_kept_rows_that_stand_already(gb):
    c = Cache(4, 2, 128, 12, [0, 5, 16, 90], 2, 90100, counts=[12, 0, 7, 1], dense=True)
    pools, args = c.dev()
    new = gb.paged_kv_keep(pools[0], pools[1], *args, new_seq_lens=torch.empty_like(args[1]))
    assert np.array_equal(bits_of(pools), c.pools)
    assert new.tolist() == [12, 5, 23, 91]


def test_more_layers_than_a_launch_takes(gb):
    c = Cache(2, 1, 64, 5, [14, 30], 300, 90200)
    pools, args = c.dev()
    new = gb.paged_kv_keep(pools[0], pools[1], *args, new_seq_lens=torch.empty_like(args[1]))
    assert np.array_equal(bits_of(pools), c.want()) and new.tolist() == (c.lens + c.counts).tolist()
    one, args = Cache(2, 1, 64, 5, [14, 30], 1, 90200).dev()
    want = Cache(2, 1, 64, 5, [14, 30], 1, 90200).want()
    gb.paged_kv_keep(one[0, 0], one[1, 0], *args)
    assert np.array_equal(bits_of(one), want)


def test_bad_requests_are_flagged_and_skipped(gb):
    def run(change, flag, skipped=(1,)):
        c = Cache(3, 2, 128, 6, [10, 20, 40], 2, 90300, counts=[5, 6, 4])
        lens, counts = c.lens.copy(), c.counts.copy()
        change(c)
        pools, args = c.dev()
        new = gb.paged_kv_keep(pools[0], pools[1], *args, new_seq_lens=torch.empty_like(args[1]))
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, flag)
        given = c.lens.copy()
        for r in skipped:
            c.lens[r], c.counts[r] = 0, 0
        assert np.array_equal(bits_of(pools), c.want())
        assert new.tolist() == [int(given[r]) if r in skipped else int(lens[r] + counts[r]) for r in range(3)]

    def put(name, at, value):
        return lambda c: getattr(c, name).__setitem__(at, value)

    for value in (-1, 10 ** 6, 2 ** 31 - 1):
        run(put("lens", 1, value), 2)
    for value in (-1, 7, 2 ** 31 - 1):
        run(put("counts", 1, value), 2)
    run(put("path", (1, 5), 500), 2)
    run(put("path", (1, 5), 2 ** 31 - 1), 2)
    run(put("path", (1, 0), -1), 16)
    run(lambda c: c.path.__setitem__((1, 3), c.path[1, 2]), 16)


def test_bad_blocks_are_flagged(gb):
    c = Cache(2, 2, 64, 6, [10, 20], 1, 90400, counts=[5, 3])
    c.path[1, :3] = [0, 7, 13]  # positions 20, 27, 33
    for bad in (-1, c.pools.shape[2], 2 ** 31 - 1):
        pools, args = c.dev()
        table = args[0].clone()
        table[1, 2] = bad  # positions 32 .. 47
        gb.paged_kv_keep(pools[0], pools[1], table, *args[1:])
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 4)
        c.counts[1] = 2  # the third row's move is left out
        same = np.array_equal(bits_of(pools), c.want())
        c.counts[1] = 3
        assert same


def test_stream_and_graph(gb):
    c = Cache(3, 2, 128, 6, [10, 20, 40], 2, 90500)
    s = torch.cuda.Stream()
    pools, args = c.dev()
    torch.cuda.synchronize()
    gb.paged_kv_keep(pools[0], pools[1], *args, stream=s)
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(pools), c.want())
    pools, args = c.dev()
    new = torch.empty_like(args[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gb.paged_kv_keep(pools[0], pools[1], *args, new_seq_lens=new)
    for _ in range(2):
        pools.copy_(torch.from_numpy(c.pools.view(np.int16)).view(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(pools), c.want()) and new.tolist() == (c.lens + c.counts).tolist()


@pytest.mark.parametrize("steps_in_graph", [False, True])
def test_steps_with_drafted_tokens(gb, steps_in_graph):
    """Three steps of append, tree attention in two layers, verification and keeping, eager and
    as a replayed graph; each step's attention against the plain form over the cache that the
    accepted tokens alone would have built."""
    S, Hq, Hkv, D, Tn, V, layers, steps = 3, 8, 2, 128, 7, 300, 2, 3
    rng = np.random.default_rng(91000)
    lens0 = [0, 13, 250]
    blocks = [-(-(n + steps * Tn) // 16) for n in lens0]
    table_h = np.full((S, max(blocks)), -1)
    at = 0
    for r, b in enumerate(blocks):
        table_h[r, :b] = np.arange(at, at + b)[::-1]
        at += b
    pools_h = synth.normal_bf16(91001, (2, layers, at, Hkv, 16, D))
    pools = torch.from_numpy(pools_h.view(np.int16).copy()).view(torch.bfloat16).cuda()
    table = to_dev_i32(table_h)
    lens, new = to_dev_i32(np.array(lens0)), to_dev_i32(np.zeros(S))
    parents_h = np.array([-1, 0, 0, 1, 1, 2, 3])
    depth = np.array([0, 1, 1, 2, 2, 2, 3])
    parents = to_dev_i32(np.tile(parents_h, (S, 1)))
    max_len = max(lens0) + steps * Tn
    inv = 1e4 ** (-np.arange(D // 2) / (D // 2))
    angle = np.arange(max_len)[:, None] * inv
    cos_sin = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().cuda()
    depth_d = to_dev_i32(depth)
    q_in = torch.empty(layers, S, Tn, Hq, D, dtype=torch.bfloat16, device="cuda")
    k_in, v_in = (torch.empty(layers, S, Tn, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    probs, drafts = (torch.empty(S, Tn, V, device="cuda") for _ in (0, 1))
    tokens, u = to_dev_i32(np.zeros((S, Tn))), torch.empty(S, Tn, device="cuda")
    o = torch.empty(layers, S, Hq, Tn, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(layers, S, Hq, Tn, device="cuda")
    q_out = torch.empty(layers, S, Hq, Tn, D, dtype=torch.bfloat16, device="cuda")
    after = torch.empty_like(pools)
    said, path, counts = (torch.empty(S, Tn, dtype=torch.int32, device="cuda") for _ in range(3))
    counts = torch.empty(S, dtype=torch.int32, device="cuda")

    def step():
        for i in range(layers):
            positions = lens[:, None] + depth_d
            gb.paged_qkv_append(q_in[i], k_in[i], v_in[i], pools[0, i], pools[1, i], table, lens,
                                cos_sin=cos_sin, positions=positions, q_out=q_out[i])
            gb.paged_attn_tree(q_out[i], pools[0, i], pools[1, i], table, lens, parents, max_len,
                               out=o[i], lse=lse[i])
        after.copy_(pools)
        gb.draft_verify(probs, drafts, tokens, parents, u, tokens_out=said, path=path, counts=counts)
        gb.paged_kv_keep(pools[0], pools[1], table, lens, path, counts, new_seq_lens=new)
        lens.copy_(new)

    def fill(s):
        gen = torch.Generator("cuda").manual_seed(s)
        for t in (q_in, k_in, v_in):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        logits = 2 * torch.randn(S, Tn, V, generator=gen, device="cuda")
        probs.copy_(logits.softmax(-1))
        drafts.copy_((logits + 0.4 * torch.randn(S, Tn, V, generator=gen, device="cuda")).softmax(-1))
        up = parents.long().clamp(min=0)
        rows = drafts.gather(1, up[:, :, None].expand(S, Tn, V)).view(-1, V)
        tokens.copy_(torch.multinomial(rows, 1, generator=gen).view(S, Tn))
        u.copy_(torch.rand(S, Tn, generator=gen, device="cuda"))

    fill(1)
    run = step
    if steps_in_graph:
        gb.paged_attn_tree(q_in[0].transpose(1, 2).contiguous(), pools[0, 0], pools[1, 0], table, lens,
                           parents, max_len)  # set-up before the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    moved = 0
    for s in range(steps):
        fill(s + 1)
        before = lens.cpu().numpy().copy()
        run()
        torch.cuda.synchronize()
        assert gb.attn_device_status() == (gb.ATTN_OK, 0)
        h = [bits_of(after[kv]) for kv in (0, 1)]
        nodes = np.full(S, Tn)
        for i in range(layers):
            want = ref.attention(bits_of(q_out[i]), h[0][i], h[1][i], table_h, before,
                                 parents.cpu().numpy(), nodes, D ** -0.5)
            keys = (before + Tn)[:, None, None].astype(np.float64)
            ref.check_attention(from_dev(o[i]), from_dev(lse[i]), want, nodes, keys)
        ph, qh, th, uh = (x.cpu().numpy() for x in (probs, drafts, tokens, u))
        paths, cs = path.cpu().numpy(), counts.cpu().numpy()
        for r in range(S):
            w_said, w_path = ref.verify_plain(ph[r], qh[r], th[r], parents_h, uh[r], Tn)
            assert paths[r, :cs[r]].tolist() == w_path and said[r, :cs[r]].tolist() == w_said
            moved += sum(i != j for j, i in enumerate(w_path))
        for kv in (0, 1):
            for i in range(layers):
                want = ref.keep(h[kv][i], table_h, before, paths, cs)
                assert np.array_equal(bits_of(pools[kv, i]), want)
        assert lens.cpu().numpy().tolist() == (before + cs).tolist()
    assert moved > 0 and lens.cpu().numpy().max() > max(lens0)
