"""draft_verify against the rule in rational numbers (small vocabularies, borders hit exactly)
and in float64 (large ones), and as a way of drawing: what it puts out follows the target."""

from __future__ import annotations

import numpy as np
import pytest

import tree_ref as ref
from gpu_util import to_dev_i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gb():
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    return gb


def dyadic(rng, *shape, bits=7):
    """Rows of multiples of 2^-bits that sum to 1, many of them 0."""
    S = np.zeros(shape, dtype=np.int64)
    rows = S.reshape(-1, shape[-1])
    for row in rows:
        np.add.at(row, (shape[-1] * rng.random(1 << bits) ** 2).astype(int), 1)
    return (S / 2.0 ** bits).astype(np.float32)


def inputs(rng, S, Tn, V, kind, p, q):
    """Tokens drawn from the draft's row of the parent (any token without a draft)."""
    parents = np.stack([ref.tree(kind, Tn, rng) for _ in range(S)])
    if kind == "random":  # one root, a few broad nodes
        parents = np.minimum((np.arange(Tn)[None] * rng.random((S, Tn)) ** 3).astype(int),
                             np.arange(Tn)[None] - 1)
    tokens = np.zeros((S, Tn), dtype=np.int64)
    for r in range(S):
        for i in range(Tn):
            row = (p if q is None else q)[r, max(parents[r, i], 0)].astype(np.float64)
            tokens[r, i] = rng.choice(V, p=row / row.sum())
    return parents, tokens


def run(gb, p, q, tokens, parents, u, nodes=None, **kw):
    f = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = gb.draft_verify(f(p), f(q), to_dev_i32(tokens), to_dev_i32(parents),
                          f(np.asarray(u, dtype=np.float32)),
                          tree_lens=None if nodes is None else to_dev_i32(nodes), **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


def check(got, want, Tn):
    out, path, counts = got
    for r, (w_out, w_path) in enumerate(want):
        assert counts[r] == len(w_path), r
        assert path[r].tolist() == w_path + [-1] * (Tn - len(w_path)), r
        assert out[r].tolist() == w_out + [-1] * (Tn - len(w_out)), r


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("kind", ["chain", "binary", "random", "star"])
@pytest.mark.parametrize("S,Tn,V", [(40, 6, 5), (20, 12, 33), (60, 3, 2), (30, 1, 9), (25, 20, 1)])
def test_rational_arithmetic(gb, drawn, kind, S, Tn, V):
    """Probabilities and random numbers are small dyadic numbers, so that borders are hit: what
    lies on one is decided as the rule says."""
    rng = np.random.default_rng(S * Tn + V + drawn)
    p = dyadic(rng, S, Tn, V)
    q = dyadic(rng, S, Tn, V) if drawn else None
    parents, tokens = inputs(rng, S, Tn, V, kind, p, q)
    u = rng.integers(0, 128, (S, Tn)) / 128
    nodes = rng.integers(0, Tn + 1, S)
    got = run(gb, p, q, tokens, parents, u, nodes)
    want = [ref.verify_exact(p[r].tolist(), None if q is None else q[r].tolist(), tokens[r],
                             parents[r], u[r].tolist(), int(nodes[r]), V) for r in range(S)]
    check(got, want, Tn)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)


def softmax_rows(rng, S, Tn, V, bf16=False):
    x = 3 * rng.standard_normal((S, Tn, V), dtype=np.float32)
    y = x + 0.7 * rng.standard_normal((S, Tn, V), dtype=np.float32)
    out = []
    for z in (x, y):
        e = np.exp(z - z.max(-1, keepdims=True))
        out.append((e / e.sum(-1, keepdims=True)).astype(np.float32))
    return out


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("S,Tn,V,kind", [(1, 8, 32000, "chain"), (3, 16, 50257, "random"),
                                         (9, 5, 511, "chain"), (4, 4, 4097, "star"),
                                         (2, 6, 131072, "binary"), (40, 7, 1000, "binary"),
                                         (1, 3, 300001, "chain"), (1, 256, 100, "random"),
                                         # fewer CTAs a request, down to one
                                         (100, 3, 20000, "star"), (300, 3, 9001, "binary"),
                                         (700, 4, 4099, "star")])
def test_large_vocabularies(gb, drawn, S, Tn, V, kind):
    rng = np.random.default_rng(V + Tn)
    p, q = softmax_rows(rng, S, Tn, V)
    parents, tokens = inputs(rng, S, Tn, V, kind, p, q)
    u = rng.random((S, Tn), dtype=np.float32)
    q = q if drawn else None
    got = run(gb, p, q, tokens, parents, u)
    want = [ref.verify_plain(p[r], None if q is None else q[r], tokens[r], parents[r], u[r], Tn)
            for r in range(S)]
    check(got, want, Tn)


@pytest.mark.parametrize("drawn", [True, False])
def test_bf16_and_strides(gb, drawn):
    """bf16 rows, and rows that are views of wider ones or shared by all nodes."""
    rng = np.random.default_rng(9)
    S, Tn, V = 6, 5, 1537
    p, q = softmax_rows(rng, S, Tn, V)
    parents, tokens = inputs(rng, S, Tn, V, "binary", p, q)
    u = rng.random((S, Tn), dtype=np.float32)
    args = [to_dev_i32(tokens), to_dev_i32(parents), torch.from_numpy(u).cuda()]
    for dtype in (torch.bfloat16, torch.float32):
        wide_p, wide_q = (torch.zeros(Tn, S, V + 3, dtype=dtype, device="cuda") for _ in (0, 1))
        vp, vq = (w[:, :, 1:V + 1].transpose(0, 1) for w in (wide_p, wide_q))
        vp.copy_(torch.from_numpy(p))
        vq.copy_(torch.from_numpy(q))
        got = [t.cpu().numpy() for t in gb.draft_verify(vp, vq if drawn else None, *args)]
        hp, hq = vp.float().cpu().numpy(), vq.float().cpu().numpy()
        check(got, [ref.verify_plain(hp[r], hq[r] if drawn else None, tokens[r], parents[r], u[r], Tn)
                    for r in range(S)], Tn)
        got = [t.cpu().numpy() for t in gb.draft_verify(
            vp[:, :1].expand(S, Tn, V), vq[:1, :1].expand(S, Tn, V) if drawn else None, *args)]
        check(got, [ref.verify_plain(np.broadcast_to(hp[r, :1], (Tn, V)),
                                     np.broadcast_to(hq[0, :1], (Tn, V)) if drawn else None,
                                     tokens[r], parents[r], u[r], Tn) for r in range(S)], Tn)


def test_the_ends_of_a_row(gb):
    """Mass at the first or last token only, at every place of a tile, and random numbers next
    to 0 and 1."""
    V = 20011
    at = [0, 1, 15, 16, 31, 32, 511, 512, 513, 4095, 4096, 8191, 20009, 20010]
    S = len(at)
    p = np.zeros((S, 2, V), dtype=np.float32)
    for r, x in enumerate(at):
        p[r, :, x] = 1
    u = np.tile(np.array([1 - 2.0 ** -24, 0.5], dtype=np.float32), (S, 1))
    u[::2, 0] = 0
    parents = np.tile([-1, 0], (S, 1))
    for drafted in (at, [x ^ 1 for x in at]):
        tokens = np.stack([np.zeros(S, dtype=int), np.array(drafted)], 1).clip(0, V - 1)
        for q in (None, np.roll(p, 1, -1)):
            got = run(gb, p, q, tokens, parents, u)
            want = [ref.verify_plain(p[r], None if q is None else q[r], tokens[r], parents[r], u[r], 2)
                    for r in range(S)]
            check(got, want, 2)
            assert all(o[c - 1] == x for o, c, x in zip(got[0], got[2], at))


def test_tokens_outside_the_vocabulary_fall(gb):
    rng = np.random.default_rng(10)
    p, q = softmax_rows(rng, 4, 3, 100)
    tokens = np.array([[0, -1, 5], [0, 100, 5], [0, 2 ** 31 - 1, -2 ** 31], [-9, 7, 5]])
    parents = np.tile([-1, 0, 0], (4, 1))
    u = np.full((4, 3), 2.0 ** -20, dtype=np.float32)
    for qq in (q, None):
        got = run(gb, p, qq, tokens, parents, u)
        assert got[1].tolist() == [[0, 2, -1], [0, 2, -1], [0, -1, -1], [0, 1, -1]]


def test_odd_probabilities(gb):
    """NaN and negative values count as 0, values above 1 as 1; a row without mass is flagged."""
    p = np.zeros((4, 1, 70), dtype=np.float32)
    p[0, 0, [3, 40]] = np.nan, 0.25
    p[1, 0, [3, 40]] = -1, 0.25
    p[2, 0, 50] = np.inf
    u = np.zeros((4, 1))
    zero = np.zeros((4, 1), dtype=int)
    got = run(gb, p, None, zero, zero - 1, u)
    assert got[0][:, 0].tolist() == [40, 40, 50, -1] and got[2].tolist() == [1, 1, 1, 1]
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 32)


def test_a_remainder_without_mass_is_left_out(gb):
    """Where the draft is above the target everywhere, a fallen child changes nothing."""
    p = np.array([[[0.25, 0.75, 0, 0]] * 3] * 3, dtype=np.float32)
    q = p.copy()
    parents = np.tile([-1, 0, 0], (3, 1))
    tokens = np.array([[0, 2, 1], [0, 2, 3], [0, 3, 0]])
    u = np.array([[0.1, 0.5, 0.9], [0.5, 0.5, 0.5], [0.9, 0.5, 0.99]])
    want = [ref.verify_exact(p[r].tolist(), q[r].tolist(), tokens[r], parents[r], u[r].tolist(), 3, 4)
            for r in range(3)]
    check(run(gb, p, q, tokens, parents, u), want, 3)
    p = np.array([[[0, 1, 0, 0]] * 3] * 3, dtype=np.float32)
    want = [ref.verify_exact(p[r].tolist(), None, [0, 1, 1], parents[r], [0.5, 1.0, 1.0], 3, 4)
            for r in range(3)]
    # (a number of 1 is outside [0, 1): the token falls although nothing else is left)
    check(run(gb, p, None, np.tile([0, 1, 1], (3, 1)), parents, np.tile([0.5, 1.0, 1.0], (3, 1))), want, 3)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_rows_that_are_no_distribution_leave_no_output_unwritten(gb, drawn, bf16):
    """Scores in the place of probabilities: sums past 4 wrap, but every token is one of the V or -1."""
    rng = np.random.default_rng(5)
    for S, Tn, V in [(7, 4, 100003), (40, 3, 4999), (9, 5, 40), (3, 2, 7)]:
        scores = [torch.from_numpy(rng.normal(0, s, (S, Tn, V)).astype(np.float32)).cuda() for s in (3, 9)]
        scores[0][0] = 1.0
        if bf16:
            scores = [x.bfloat16() for x in scores]
        parents = np.tile(np.arange(Tn) - 1, (S, 1))
        tokens = rng.integers(0, V, (S, Tn))
        for u in (0.0, 0.3, 0.999):
            outs = [torch.full((S, Tn), 1 << 30, dtype=torch.int32, device="cuda") for _ in range(2)]
            counts = torch.full((S,), 1 << 30, dtype=torch.int32, device="cuda")
            gb.draft_verify(scores[0], scores[1] if drawn else None, to_dev_i32(tokens), to_dev_i32(parents),
                            torch.full((S, Tn), u, device="cuda"), tokens_out=outs[0], path=outs[1],
                            counts=counts)
            out, path, counts = (t.cpu().numpy() for t in (*outs, counts))
            assert (out >= -1).all() and (out < V).all()
            assert (path >= -1).all() and (path < Tn).all()
            assert (counts >= 1).all() and (counts <= Tn).all()
    status, flags = gb.attn_device_status()
    assert flags in (0, 32)


def test_bad_trees_and_sizes_are_flagged(gb):
    rng = np.random.default_rng(11)
    p, q = softmax_rows(rng, 3, 4, 50)
    tokens, u = np.zeros((3, 4), dtype=int), np.full((3, 4), 0.5)
    parents = np.tile([-1, 0, 1, 2], (3, 1))
    good = run(gb, p, q, tokens, parents, u)
    for where, value in (((1, 0), 0), ((1, 2), 2), ((1, 3), -2), ((1, 1), 2 ** 31 - 1)):
        bad = parents.copy()
        bad[where] = value
        got = run(gb, p, q, tokens, bad, u)
        assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 16)
        assert got[2][1] == 0 and (got[0][1] == -1).all() and (got[1][1] == -1).all()
        assert all((a[[0, 2]] == b[[0, 2]]).all() for a, b in zip(got, good))
    for n in (-1, 5, 2 ** 31 - 1):
        got = run(gb, p, q, tokens, parents, u, np.array([4, n, 4]))
        assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2)
        assert got[2][1] == 0 and all((a[[0, 2]] == b[[0, 2]]).all() for a, b in zip(got, good))


def test_no_nodes_at_all(gb):
    p = torch.zeros(3, 0, 10, device="cuda")
    i = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    counts = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    out, path, c = gb.draft_verify(p, None, i, i, torch.zeros(3, 0, device="cuda"), counts=counts)
    assert out.shape == path.shape == (3, 0) and c is counts and c.tolist() == [0, 0, 0]


def test_given_outputs_graph_and_stream(gb):
    rng = np.random.default_rng(12)
    S, Tn, V = 5, 6, 9001
    p, q = softmax_rows(rng, S, Tn, V)
    parents, tokens = inputs(rng, S, Tn, V, "random", p, q)
    u = rng.random((S, Tn), dtype=np.float32)
    want = run(gb, p, q, tokens, parents, u)
    args = [torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda(), to_dev_i32(tokens),
            to_dev_i32(parents), torch.from_numpy(u).cuda()]
    big = torch.full((2, S + 2, Tn), 55, dtype=torch.int32, device="cuda")
    counts = torch.full((S + 2,), 55, dtype=torch.int32, device="cuda")
    kw = dict(tokens_out=big[0, 1:-1], path=big[1, 1:-1], counts=counts[1:-1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gb.draft_verify(*args, stream=s, **kw)
    torch.cuda.synchronize()
    assert all((a.cpu().numpy() == b).all() for a, b in zip(got, want))
    assert (big[:, [0, -1]] == 55).all() and (counts[[0, -1]] == 55).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gb.draft_verify(*args, **kw)
    for _ in range(3):
        big.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all((a.cpu().numpy() == b).all() for a, b in zip(got, want))


@pytest.mark.parametrize("drawn", [True, False])
def test_outputs_in_the_place_of_inputs(gb, drawn):
    rng = np.random.default_rng(21)
    S, Tn, V = 50, 9, 5003
    p, q = softmax_rows(rng, S, Tn, V)
    q = q if drawn else None
    parents, tokens = inputs(rng, S, Tn, V, "random", p, q)
    u = rng.random((S, Tn), dtype=np.float32)
    nodes = rng.integers(0, Tn + 1, S)
    want = run(gb, p, q, tokens, parents, u, nodes)
    t, pa, n = to_dev_i32(tokens), to_dev_i32(parents), to_dev_i32(nodes)
    got = gb.draft_verify(torch.from_numpy(p).cuda(), None if q is None else torch.from_numpy(q).cuda(), t, pa,
                          torch.from_numpy(u).cuda(), tree_lens=n, tokens_out=t, path=pa, counts=n)
    assert got[0] is t and got[1] is pa and got[2] is n
    assert all((a.cpu().numpy() == b).all() for a, b in zip(got, want))


def test_calls_on_two_streams_at_once(gb):
    rng = np.random.default_rng(22)
    sets, want = [], []
    for S, Tn, V, kind, drawn in [(3, 8, 100003, "chain", True), (200, 5, 4001, "star", False),
                                  (20, 12, 20000, "random", True)]:
        p, q = softmax_rows(rng, S, Tn, V)
        parents, tokens = inputs(rng, S, Tn, V, kind, p, q)
        u = rng.random((S, Tn), dtype=np.float32)
        want.append(run(gb, p, q if drawn else None, tokens, parents, u))
        sets.append([torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda() if drawn else None,
                     to_dev_i32(tokens), to_dev_i32(parents), torch.from_numpy(u).cuda()])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[gb.draft_verify(*a, stream=s) for a in sets] for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for outs in got:
        for g, w in zip(outs, want):
            assert all((a.cpu().numpy() == b).all() for a, b in zip(g, w))


@pytest.mark.parametrize("drawn", [True, False])
def test_tokens_follow_the_target(gb, drawn):
    """Over many requests with numbers of their own, the first token put out is distributed as
    the target's row: 2^17 draws, each frequency within 5.5 standard deviations (a false alarm
    in about one run of a million)."""
    S, V = 1 << 17, 6
    gen = torch.Generator("cuda").manual_seed(3)
    p0 = torch.tensor([0.3, 0.05, 0.25, 0.2, 0.0, 0.2], device="cuda")
    q0 = torch.tensor([0.1, 0.4, 0.1, 0.2, 0.1, 0.1], device="cuda")
    Tn = 4  # three children of the root
    p, q = (x.expand(S, Tn, V) for x in (p0, q0))
    if drawn:
        tokens = torch.multinomial(q0, S * Tn, replacement=True, generator=gen).view(S, Tn).int()
    else:
        tokens = torch.tensor([0, 1, 0, 3], device="cuda").int().repeat(S, 1)
    parents = torch.tensor([-1, 0, 0, 0], device="cuda").int().repeat(S, 1)
    u = torch.rand(S, Tn, generator=gen, device="cuda")
    out, _, counts = gb.draft_verify(p, q if drawn else None, tokens, parents, u)
    freq = torch.bincount(out[:, 0].long(), minlength=V).double() / S
    sd = (p0.double() * (1 - p0.double()) / S).sqrt()
    assert ((freq - p0.double()).abs() <= 5.5 * sd + 1e-12).all(), freq
    assert (counts == 2).double().mean() > (0.5 if drawn else 0.4)
