"""qkv_norm_rope, its gradients and the appends built on it (bf16 and 4 bits) against
float64 references.

Tolerances.  A result is rounded to bf16 once: half a step, 2^-8 of the value.  Before
that, fp32: the sum of D squares (8 in a row, then 4 levels), its mean, rsqrt (2 steps)
and two products are within 2^-20 of the normed value; the rotation adds two products
and a sum, each 2^-24 of at most sqrt(2) row maxima.  So 2^-18 of the row's largest
magnitude covers the forward pass.  The backward pass adds a dot product of the same
form and a difference of terms no larger than 3 row maxima of r * w * g: 2^-16 of the
largest |r w| times the largest |g| of the row.  A weight gradient is a sum of n terms
in chains whose joined length is below 64 + n / 3648 / 2; each link loses 2^-24 of the
sum of magnitudes, and each term carries 2^-19.
"""

from __future__ import annotations

import numpy as np
import pytest

import rope_ref as ref
import synth
from gpu_util import bits_of, from_dev, to_dev, to_dev_i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = 2.0 ** -8


@pytest.fixture(params=["compiled binding", "Python binding"])
def gb(request, monkeypatch):
    import attention_flashattention_fwd_03_gb300 as gb
    gb.lib()
    gb._load_torch()
    if request.param == "Python binding":
        monkeypatch.setattr(gb, "_quick", None)
    elif gb._quick is None:
        pytest.fail("_binding was not built")
    return gb


class Case:
    def __init__(self, B, T, Hq, Hkv, D, rot, norm, interleaved, seed, start=0, explicit=True):
        self.B, self.T, self.Hq, self.Hkv, self.D, self.rot = B, T, Hq, Hkv, D, rot
        self.interleaved = interleaved
        self.rows = synth.normal_bf16(seed, (B, T, Hq + 2 * Hkv, D), 2.0)  # a fused projection
        self.fused = to_dev(self.rows)
        self.q, self.k, self.v = self.fused.split([Hq, Hkv, Hkv], 2)
        self.wb = [synth.float_to_bf16_bits((1 + 0.2 * synth.normals(seed + i, D)).astype(np.float32))
                   for i in (1, 2)] if norm else [None, None]
        self.wq, self.wk = (to_dev(w) if norm else None for w in self.wb)
        self.pos = start + np.arange(B)[:, None] * 3 + np.arange(T)[None]
        if not explicit:
            self.pos = np.broadcast_to(np.arange(T), (B, T))
        self.table = ref.table(int(self.pos.max()) + 1 + 64, rot) if rot else None
        self.cs = torch.from_numpy(self.table).cuda() if rot else None
        self.positions = to_dev_i32(self.pos) if explicit and rot else None
        self.how = dict(cos_sin=self.cs, q_weight=self.wq, k_weight=self.wk, eps=ref.EPS,
                        interleaved=interleaved)

    def x(self, i):
        cut = np.split(self.rows, [self.Hq, self.Hq + self.Hkv], 2)[i]
        return synth.bf16_bits_to_float(cut).astype(np.float64)

    def w(self, i):
        return None if self.wb[i] is None else synth.bf16_bits_to_float(self.wb[i]).astype(np.float64)

    def rows_of_table(self, pos=None):
        return None if self.table is None else self.table[self.pos if pos is None else pos]

    def expect(self, i, pos=None):
        return ref.norm_rope(self.x(i), self.w(i), self.rows_of_table(pos), self.interleaved)


def close_rows(got, want):
    """[B, H, T, D] against [B, T, H, D]."""
    want = want.transpose(0, 2, 1, 3)
    tol = HALF * np.abs(want) + 2.0 ** -18 * np.abs(want).max(-1, keepdims=True)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


CASES = [
    # B, T, Hq, Hkv, D, rot, norm, interleaved, start, explicit positions
    (1, 1, 1, 1, 128, 128, True, False, 0, False),
    (2, 5, 12, 2, 128, 128, True, False, 1000, True),
    (3, 77, 4, 2, 64, 64, True, True, 0, True),
    (1, 130, 7, 1, 64, 32, False, False, 5, True),
    (2, 33, 3, 3, 128, 24, True, False, 0, False),
    (1, 40, 5, 5, 128, 40, False, True, 9, True),
    (4, 9, 2, 1, 64, 8, True, True, 0, False),
    (1, 300, 32, 8, 128, 128, True, False, 50000, True),
    (2, 6, 4, 2, 64, 0, True, False, 0, False),
    (2, 6, 4, 2, 128, 0, False, False, 0, False),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,norm,il,start,explicit", CASES)
def test_forward(gb, B, T, Hq, Hkv, D, rot, norm, il, start, explicit):
    c = Case(B, T, Hq, Hkv, D, rot, norm, il, 31000 + T, start, explicit)
    q, k, v = gb.qkv_norm_rope(c.q, c.k, c.v, positions=c.positions, **c.how)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    close_rows(from_dev(q), c.expect(0))
    close_rows(from_dev(k), c.expect(1))
    assert torch.equal(v, c.v.transpose(1, 2))
    # each operand alone, from other layouts, gives the same bits
    q1, none, _ = gb.qkv_norm_rope(c.q.contiguous(), None, positions=c.positions, **c.how)
    kt = c.k.transpose(1, 2).contiguous().transpose(1, 2)
    _, k1, _ = gb.qkv_norm_rope(None, kt, positions=c.positions, **c.how)
    _, none2, v1 = gb.qkv_norm_rope(None, None, c.v.contiguous(), positions=c.positions, **c.how)
    assert none is None and none2 is None
    assert torch.equal(q, q1) and torch.equal(k, k1) and torch.equal(v, v1)


@pytest.mark.parametrize("D,rot,il", [(128, 128, False), (64, 64, False), (128, 40, False),
                                      (64, 64, True), (128, 32, True)])
def test_rotation_rounds_every_operation(gb, D, rot, il):
    """Without a norm the rows are what eager fp32 operations give, bit for bit."""
    c = Case(3, 50, 5, 2, D, rot, False, il, 66000 + rot, 7)
    cs = c.cs[c.positions.long()][:, :, None]
    cos, sin = cs.chunk(2, -1)
    for x, y in zip((c.q, c.k), gb.qkv_norm_rope(c.q, c.k, positions=c.positions, **c.how)):
        r = x[..., :rot].float()
        a, b = (r[..., 0::2], r[..., 1::2]) if il else r.chunk(2, -1)
        want = (a * cos - b * sin, b * cos + a * sin)
        want = torch.stack(want, -1).flatten(-2) if il else torch.cat(want, -1)
        want = torch.cat([want.bfloat16(), x[..., rot:]], -1)
        assert torch.equal(y, want.transpose(1, 2))


@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,norm,il,start,explicit", CASES)
def test_backward(gb, B, T, Hq, Hkv, D, rot, norm, il, start, explicit):
    c = Case(B, T, Hq, Hkv, D, rot, norm, il, 32000 + T, start, explicit)
    gbits = [synth.normal_bf16(33000 + i, (B, h, T, D)) for i, h in enumerate((Hq, Hkv, Hkv))]
    g = [to_dev(x) for x in gbits]
    dq, dk, dv, dwq, dwk = gb.qkv_norm_rope_bwd(*g, c.q, c.k, positions=c.positions, **c.how)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert torch.equal(dv, g[2].transpose(1, 2))
    assert dq.data_ptr() == dk.data_ptr() - 2 * Hq * D  # one fused buffer
    for i, (d, dw) in enumerate(((dq, dwq), (dk, dwk))):
        gf = synth.bf16_bits_to_float(gbits[i]).astype(np.float64).transpose(0, 2, 1, 3)
        x, w = c.x(i), c.w(i)
        want, ww, mags = ref.norm_rope_bwd(gf, x, w, c.rows_of_table(), il)
        size = np.abs(gf).max(-1, keepdims=True)
        if norm:
            size = size * np.abs(w).max() / np.sqrt((x * x).mean(-1, keepdims=True) + ref.EPS)
        tol = HALF * np.abs(want) + 2.0 ** -16 * size
        assert np.all(np.abs(from_dev(d) - want) <= tol)
        if not norm:
            assert dw is None
            continue
        n = B * T * (Hq, Hkv)[i]
        tol = ((64 + n / 3648 / 2) * 2.0 ** -24 + 2.0 ** -19) * mags
        assert np.all(np.abs(from_dev(dw) - ww) <= tol)
    # given buffers and operands left out (the weight gradient's order of summation goes
    # by which operands take part, so its bits are compared between equal calls only)
    buf = torch.full((B, T, Hkv + 3, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = gb.qkv_norm_rope_bwd(None, g[1], None, None, c.k, positions=c.positions,
                               dk=buf[:, :, 1:1 + Hkv], cos_sin=c.cs, k_weight=c.wk,
                               interleaved=il)
    assert out[0] is None and out[2] is None and out[3] is None
    assert torch.equal(buf[:, :, 1:1 + Hkv], dk)
    assert torch.all(buf[:, :, 0] == 7) and torch.all(buf[:, :, 1 + Hkv:] == 7)
    if norm:
        n = B * T * Hkv
        tol = ((64 + n / 3648 / 2) * 2.0 ** -24 + 2.0 ** -19) * mags
        assert np.all(np.abs(from_dev(out[4]) - ww) <= tol)


def test_many_tokens_share_the_weight_gradient(gb):
    """More tokens than the backward grid has warps, so every CTA takes several."""
    c = Case(2, 4000, 3, 1, 64, 64, True, False, 34000, 0, False)
    g = [synth.normal_bf16(34100 + i, (2, h, 4000, 64)) for i, h in enumerate((3, 1))]
    args = (to_dev(g[0]), to_dev(g[1]), None, c.q, c.k)
    out = gb.qkv_norm_rope_bwd(*args, **c.how)
    again = gb.qkv_norm_rope_bwd(*args, **c.how)
    for i in (0, 1):
        gf = synth.bf16_bits_to_float(g[i]).astype(np.float64).transpose(0, 2, 1, 3)
        _, ww, mags = ref.norm_rope_bwd(gf, c.x(i), c.w(i), c.rows_of_table(), False)
        n = 8000 * (3, 1)[i]
        tol = ((64 + n / 3648 / 2) * 2.0 ** -24 + 2.0 ** -19) * mags
        assert np.all(np.abs(from_dev(out[3 + i]) - ww) <= tol)
        assert torch.equal(out[3 + i], again[3 + i]) and torch.equal(out[i], again[i])


def test_empty_batches(gb):
    q = torch.empty((2, 0, 4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, _, _ = gb.qkv_norm_rope(q, None, q_weight=w)
    assert y.shape == (2, 4, 0, 64)
    out = gb.qkv_norm_rope_bwd(y, None, None, q, None, q_weight=w)
    assert out[0].shape == q.shape and torch.all(out[3] == 0)


def test_repeated_input_and_zero_rows(gb):
    """A broadcast input (stride 0) and rows of zeros (the norm divides by sqrt(eps))."""
    one = to_dev(synth.normal_bf16(35000, (1, 1, 2, 64)))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, _, _ = gb.qkv_norm_rope(one.expand(3, 5, 2, 64), None, q_weight=w)
    assert torch.equal(y, y[:1, :, :1].expand(3, 2, 5, 64))
    z, _, _ = gb.qkv_norm_rope(torch.zeros_like(one), None, q_weight=w)
    assert torch.all(z == 0)


def test_positions_outside_the_table(gb):
    c = Case(2, 3, 2, 1, 64, 64, True, False, 36000, 0, True)
    pos = torch.tensor([[0, -1, 2], [3, 4, len(c.table)]], dtype=torch.int32, device="cuda")
    q, k, v = gb.qkv_norm_rope(c.q, c.k, c.v, positions=pos, **c.how)
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 8)
    bad = torch.tensor([[0, 1, 0], [0, 0, 1]], dtype=torch.bool, device="cuda")
    for y, i in ((q, 0), (k, 1)):
        rows = y.transpose(1, 2)
        assert torch.all(rows[bad].isnan()) and not torch.any(rows[~bad].isnan())
    assert torch.equal(v, c.v.transpose(1, 2))
    out = gb.qkv_norm_rope_bwd(q * 0 + 1, k * 0 + 1, None, c.q, c.k, positions=pos, **c.how)
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 8)
    assert torch.all(out[0][bad].isnan()) and torch.all(out[3].isnan()) and torch.all(out[4].isnan())


def test_another_stream_and_a_replayed_graph(gb):
    c = Case(2, 50, 4, 2, 128, 128, True, False, 37000, 0, False)
    want = gb.qkv_norm_rope(c.q, c.k, c.v, **c.how)
    g = [torch.ones_like(t) for t in want]
    dwant = gb.qkv_norm_rope_bwd(*g, c.q, c.k, **c.how)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = gb.qkv_norm_rope(c.q, c.k, c.v, stream=s, **c.how)
    dgot = gb.qkv_norm_rope_bwd(*g, c.q, c.k, stream=s, **c.how)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + dwant, got + dgot))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = gb.qkv_norm_rope(c.q, c.k, c.v, **c.how)
        dgot = gb.qkv_norm_rope_bwd(*g, c.q, c.k, **c.how)
    for _ in range(2):
        for t in got + dgot:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want + dwant, got + dgot))


# --------------------------------------------------------------------------- #
# appends
# --------------------------------------------------------------------------- #
def table_for(lens, Tn, seed, spare=3, max_blocks=None):
    blocks = [-(-(n + Tn) // 16) for n in lens]
    perm = synth.permutation(seed, sum(blocks) + spare)
    bt = np.full((len(lens), max_blocks or max(max(blocks), 1)), -1, np.int32)
    at = 0
    for r, n in enumerate(blocks):
        bt[r, :n] = perm[at:at + n]
        at += n
    return bt, len(perm)


def scatter(pool, bt, lens, rows, r0=0):
    """Host scatter of rows [S, Hkv, Tn, D] (bits) into a bf16 pool's bits."""
    for r in range(rows.shape[0]):
        for t in range(rows.shape[2]):
            p = lens[r] + t
            pool[bt[r, p // 16], :, p % 16] = rows[r, :, t]


APPENDS = [
    # lens, Tn, Hq, Hkv, D, rot, norm, interleaved, explicit positions
    ([0, 1, 15, 16, 17, 511, 4095], 1, 12, 2, 128, 128, True, False, False),
    ([0, 31, 32, 100], 5, 4, 4, 64, 64, True, True, True),
    ([7, 0], 37, 3, 1, 64, 32, False, False, False),
    ([250], 300, 8, 2, 128, 24, True, False, True),
    ([3, 20], 2, 6, 3, 128, 0, False, False, False),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,il,ops", [
    (600, 3, 9, 1, 128, False, "qkv"),   # more tokens than warps, T far below a warp's stride
    (2500, 1, 3, 2, 64, True, "qkv"),
    (2, 1500, 17, 2, 64, False, "qkv"),  # rows behind the last full pass
    (3, 811, 33, 1, 128, True, "qk"),    # T of the very stride of the warps
    (1, 2000, 8, 20, 128, False, "kv"),
    (700, 2, 16, 4, 128, False, "q"),
    (5, 400, 1, 24, 64, False, "v"),
])
def test_backward_of_many_tokens(gb, B, T, Hq, Hkv, D, il, ops):
    """Warps that take many tokens, of all, two and one of the operands."""
    c = Case(B, T, Hq, Hkv, D, D, True, il, 64000 + T)
    bits = [synth.normal_bf16(65000 + i, (B, h, T, D)) for i, h in enumerate((Hq, Hkv, Hkv))]
    g = [to_dev(x) if o in ops else None for x, o in zip(bits, "qkv")]
    how = dict(c.how, q_weight=c.wq if "q" in ops else None, k_weight=c.wk if "k" in ops else None)
    out = gb.qkv_norm_rope_bwd(*g, c.q, c.k, positions=c.positions, **how)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    assert [x is not None for x in out] == [o in ops for o in "qkvqk"]
    if "v" in ops:
        assert torch.equal(out[2], g[2].transpose(1, 2))
    for i, o in enumerate("qk"):
        if o not in ops:
            continue
        gf = synth.bf16_bits_to_float(bits[i]).astype(np.float64).transpose(0, 2, 1, 3)
        x, w = c.x(i), c.w(i)
        want, ww, mags = ref.norm_rope_bwd(gf, x, w, c.rows_of_table(), il)
        size = np.abs(gf).max(-1, keepdims=True)
        size = size * np.abs(w).max() / np.sqrt((x * x).mean(-1, keepdims=True) + ref.EPS)
        assert np.all(np.abs(from_dev(out[i]) - want) <= HALF * np.abs(want) + 2.0 ** -16 * size)
        # a lane adds its share of the rows, then at most 32 rows of a CTA, 10 CTAs and 32 sums
        # follow, each addition off by half a step of the sum so far
        share = (B * T // 810 + 1) * ((Hq, Hkv)[i] * D // 256 + 1)
        tol = ((share + 32 + 10 + 32) * 2.0 ** -24 + 2.0 ** -19) * mags
        assert np.all(np.abs(from_dev(out[3 + i]) - ww) <= tol)


def test_no_gradient_is_lost_without_a_word(gb):
    """Calls through which torch expects a derivative are refused by both bindings; the same
    operands under no_grad, and in an autograd.Function, give what they give without."""
    c = Case(2, 5, 4, 2, 64, 64, True, False, 47000)
    good = gb.qkv_norm_rope(c.q, c.k, c.v, positions=c.positions, **c.how)
    g = [torch.ones_like(x) for x in good]
    good_bwd = gb.qkv_norm_rope_bwd(*g, c.q, c.k, positions=c.positions, **c.how)
    wq, wk = (torch.nn.Parameter(c.how[n]) for n in ("q_weight", "k_weight"))
    how = dict(c.how, positions=c.positions, q_weight=wq, k_weight=wk)
    with pytest.raises(ValueError, match="records nothing"):
        gb.qkv_norm_rope(c.q, c.k, c.v, **how)
    with pytest.raises(ValueError, match="records nothing"):
        gb.qkv_norm_rope_bwd(*g, c.q, c.k, **how)
    x = c.q.clone().requires_grad_()
    with pytest.raises(ValueError, match="records nothing"):
        gb.qkv_norm_rope(x * 1, c.k, c.v, positions=c.positions, **c.how)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(c.q, torch.ones_like(c.q))
        with pytest.raises(ValueError, match="records nothing"):
            gb.qkv_norm_rope(dual, c.k, c.v, positions=c.positions, **c.how)
    with torch.no_grad():
        for a, b in zip(good, gb.qkv_norm_rope(c.q, c.k, c.v, **how)):
            assert torch.equal(a, b)
        for a, b in zip(good_bwd, gb.qkv_norm_rope_bwd(*g, c.q, c.k, **how)):
            assert torch.equal(a, b)

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, w, wk):
            ctx.save_for_backward(q, k, w, wk)
            return gb.qkv_norm_rope(q, k, None, positions=c.positions,
                                    **dict(c.how, q_weight=w, k_weight=wk))[:2]

        @staticmethod
        def backward(ctx, dq, dk):
            q, k, w, wk = ctx.saved_tensors
            dq, dk, _, dw, dwk = gb.qkv_norm_rope_bwd(
                dq.contiguous(), dk.contiguous(), None, q, k, positions=c.positions,
                **dict(c.how, q_weight=w, k_weight=wk))
            return dq, dk, dw.to(w.dtype), dwk.to(wk.dtype)

    k = c.k.clone().requires_grad_()
    q1, k1 = Turn.apply(x, k, wq, wk)
    assert torch.equal(q1, good[0]) and torch.equal(k1, good[1])
    torch.autograd.backward([q1, k1], g[:2])
    same = gb.qkv_norm_rope_bwd(*g[:2], None, c.q, c.k, positions=c.positions, **c.how)
    assert torch.equal(x.grad, same[0]) and torch.equal(k.grad, same[1])
    assert torch.equal(wq.grad, same[3].bfloat16()) and torch.equal(wk.grad, same[4].bfloat16())


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("lens,Tn,Hq,Hkv,D,rot,norm,il,explicit", APPENDS)
def test_append_matches_the_forward_bit_for_bit(gb, four, lens, Tn, Hq, Hkv, D, rot, norm, il,
                                                explicit):
    S = len(lens)
    c = Case(S, Tn, Hq, Hkv, D, rot, norm, il, 38000 + Tn, 0, explicit)
    cached = np.array(lens)[:, None] + np.arange(Tn)[None]
    pos = c.pos if explicit else cached
    if rot:
        c.table = ref.table(int(pos.max()) + 1, rot)
        c.how["cos_sin"] = torch.from_numpy(c.table).cuda()
    q0, k0, v0 = gb.qkv_norm_rope(c.q, c.k, c.v, positions=to_dev_i32(pos) if rot else None, **c.how)
    bt, NB = table_for(lens, Tn, 39)
    before, after = to_dev_i32(np.array(lens)), torch.full((S,), -5, dtype=torch.int32, device="cuda")
    how = dict(c.how, positions=c.positions, new_seq_lens=after)
    start = synth.normal_bf16(38500, (2, NB, Hkv, 16, D))
    scatter_to = start.copy()
    scatter(scatter_to[0], bt, lens, bits_of(k0))
    scatter(scatter_to[1], bt, lens, bits_of(v0))
    if four:
        pool = torch.from_numpy(ref.pool_from_bf16(*start)).cuda()
        q, new = gb.paged_kv4_append(c.q, c.k, c.v, pool, to_dev_i32(bt), before, **how)
        torch.cuda.synchronize()
        # untouched chunks keep every byte, written tokens hold the reference's bytes
        assert np.array_equal(pool.cpu().numpy(), ref.pool_from_bf16(*scatter_to))
    else:
        kp, vp = to_dev(start[0]), to_dev(start[1])
        q, new = gb.paged_qkv_append(c.q, c.k, c.v, kp, vp, to_dev_i32(bt), before, **how)
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(kp), scatter_to[0])
        assert np.array_equal(bits_of(vp), scatter_to[1])
    assert torch.equal(q, q0) and new is after
    assert after.cpu().tolist() == [n + Tn for n in lens]
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    close_rows(from_dev(q), c.expect(0, pos))


@pytest.mark.parametrize("four", [False, True])
def test_append_bad_requests_are_flagged_and_skipped(gb, four):
    lens, Hkv, D = [10, 20, 30, 40, 5], 2, 64
    c = Case(5, 1, 4, Hkv, D, 64, True, False, 40000)
    bt, NB = table_for(lens, 1, 41)
    bt[1, 20 // 16] = NB + 2                       # a block outside the pool
    bad = np.array([10, 20, bt.shape[1] * 16, 40, -1])  # 2: no room, 4: no length
    cs = torch.from_numpy(ref.table(40, 64)).cuda()     # 3: position 40 is outside
    start = synth.normal_bf16(40500, (2, NB, Hkv, 16, D))
    after = torch.full((5,), -9, dtype=torch.int32, device="cuda")
    how = dict(c.how, cos_sin=cs, new_seq_lens=after)
    _, k0, v0 = gb.qkv_norm_rope(c.q[:1], c.k[:1], c.v[:1],
                                 positions=to_dev_i32(np.array([[10]])), **dict(c.how, cos_sin=cs))
    scatter_to = start.copy()
    scatter(scatter_to[0], bt, [10], bits_of(k0))
    scatter(scatter_to[1], bt, [10], bits_of(v0))
    if four:
        pool = torch.from_numpy(ref.pool_from_bf16(*start)).cuda()
        q, _ = gb.paged_kv4_append(c.q, c.k, c.v, pool, to_dev_i32(bt), to_dev_i32(bad), **how)
        torch.cuda.synchronize()
        assert np.array_equal(pool.cpu().numpy(), ref.pool_from_bf16(*scatter_to))
    else:
        kp, vp = to_dev(start[0]), to_dev(start[1])
        q, _ = gb.paged_qkv_append(c.q, c.k, c.v, kp, vp, to_dev_i32(bt), to_dev_i32(bad), **how)
        torch.cuda.synchronize()
        assert np.array_equal(bits_of(kp), scatter_to[0])
        assert np.array_equal(bits_of(vp), scatter_to[1])
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2 | 4 | 8)
    assert after.cpu().tolist() == [11, 21, bt.shape[1] * 16, 41, -1]
    nan = torch.isnan(q).flatten(1).all(1).cpu().tolist()
    assert nan == [False, False, True, True, True]


@pytest.mark.parametrize("four", [False, True])
def test_append_of_no_tokens_keeps_the_lengths(gb, four):
    c = Case(3, 1, 4, 2, 64, 64, True, False, 40900)
    none = [x[:, :0] for x in (c.q, c.k, c.v)]
    bt, NB = table_for([4, 9, 20], 1, 42)
    pools = [torch.full((NB, 2, 18 * 64), 3, dtype=torch.uint8, device="cuda")] if four else [
        torch.full((NB, 2, 16, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    lens, new = to_dev_i32(np.array([4, 9, 20])), torch.full((3,), -9, dtype=torch.int32, device="cuda")
    op = gb.paged_kv4_append if four else gb.paged_qkv_append
    table = to_dev_i32(bt)
    q, after = op(*none, *pools, table, lens, new_seq_lens=new, **c.how)
    torch.cuda.synchronize()
    assert q.shape == (3, 4, 0, 64) and after is new and torch.equal(new, lens)
    assert all(torch.all(p == 3) for p in pools)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        op(*none, *pools, table, lens, new_seq_lens=new, **c.how)
    lens += 7
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(new, lens)


def test_append_without_queries(gb):
    c = Case(2, 3, 1, 2, 128, 128, True, False, 41000)
    bt, NB = table_for([4, 9], 3, 42)
    pools = [torch.zeros((NB, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    lens = to_dev_i32(np.array([4, 9]))
    q, _ = gb.paged_qkv_append(c.q, c.k, c.v, *pools[:2], to_dev_i32(bt), lens, **c.how)
    none, new = gb.paged_qkv_append(None, c.k, c.v, *pools[2:], to_dev_i32(bt), lens, **c.how)
    assert q is not None and none is None and new is None
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.parametrize("D", [64, 128])
def test_quantiser_edges(gb, D):
    """Zeros, NaN, infinities, the largest and smallest magnitudes, and exact ties."""
    x = np.zeros((12, 1, 1, D), np.float32)
    x[1, ..., 3] = np.nan
    x[2, ..., 33] = np.inf
    x[3, ..., 5] = -np.inf
    x[4] = 3.3e38 * np.where(np.arange(D) % 2, 1, -1)
    x[5] = 1e-39 * np.arange(D)
    x[6] = 2e-38 * synth.normals(5, D)
    x[7] = 0.5 * np.arange(D) % 7.5  # scale 1: values at half steps
    x[7, ..., ::32] = 7
    x[8] = -x[7]
    x[9] = np.arange(D) - 40
    x[10] = 1e6 * synth.normals(6, D)
    x[11] = np.exp(4 * synth.normals(7, D))
    bits = synth.float_to_bf16_bits(x)
    t = to_dev(bits)
    lens = to_dev_i32(np.zeros(12))
    bt = to_dev_i32(np.arange(12)[:, None])
    pool = torch.randint(0, 256, (12, 1, 18 * D), dtype=torch.uint8, device="cuda")
    want = pool.cpu().numpy()
    for r in range(12):
        ref.write_pool(want, r, 0, 0, bits[r, 0, 0], bits[r, 0, 0])
    gb.paged_kv4_append(None, t, t, pool, bt, lens)
    assert np.array_equal(pool.cpu().numpy(), want)
    k, v = gb.paged_kv4_gather(pool, bt, lens + 1, 1)
    assert torch.equal(k.isnan(), v.isnan()) and torch.equal(k.nan_to_num(), v.nan_to_num())
    vals = ref.values(*ref.quantise(bits[:, 0]))
    assert np.array_equal(from_dev(k)[:, 0], vals, equal_nan=True)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)


# --------------------------------------------------------------------------- #
# gather
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 2)])
def test_gather_returns_the_values_and_leaves_the_rest(gb, D, Hkv):
    lens = [0, 1, 15, 16, 17, 200, 333]
    bt, NB = table_for(lens, 0, 43)
    kb, vb = synth.normal_bf16(42000, (2, NB, Hkv, 16, D))
    pool = torch.from_numpy(ref.pool_from_bf16(kb, vb)).cuda()
    M = 340
    out = [torch.full((len(lens), Hkv, M, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    gb.paged_kv4_gather(pool, to_dev_i32(bt), to_dev_i32(np.array(lens)), M, *out)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    for o, bits in zip(out, (kb, vb)):
        got, want = bits_of(o), ref.value_bits(bits)
        for r, n in enumerate(lens):
            t = np.arange(n)
            assert np.array_equal(got[r, :, :n], want[bt[r, t // 16], :, t % 16].transpose(1, 0, 2))
        assert all(torch.all(o[r, :, n:] == 9) for r, n in enumerate(lens))


def test_gather_flags_bad_requests(gb):
    lens, D = [20, 33, 40], 64
    bt, NB = table_for(lens, 0, 44)
    bt[1, 1] = -1
    kb, vb = synth.normal_bf16(43000, (2, NB, 1, 16, D))
    pool = torch.from_numpy(ref.pool_from_bf16(kb, vb)).cuda()
    bad = to_dev_i32(np.array([20, 33, 41]))
    k, v = gb.paged_kv4_gather(pool, to_dev_i32(bt), bad, 40)
    assert gb.attn_device_status() == (gb.ATTN_ERR_DEVICE, 2 | 4)
    for o in (k, v):
        assert not o[0].isnan().any() and torch.all(o[2] == 0)
        nan = o[1, 0].isnan().all(-1).cpu().numpy()
        assert np.array_equal(np.nonzero(nan)[0], np.arange(16, 32))
