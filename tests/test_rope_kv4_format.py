"""The 4-bit cache's format and the norm + rotation formulas on the CPU: what the
references the GPU tests use must satisfy, and the argument checks of the entry points."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import attention_flashattention_fwd_03_gb300 as gb
import rope_ref as ref
import synth

A16 = 0x100000  # an aligned address that no check dereferences


# --------------------------------------------------------------------------- #
# format
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("per", [8, 4])
def test_every_channel_has_a_nibble_of_its_own(D, per):
    assert sorted(ref.nibble(c, D, per) for c in range(D)) == list(range(D))


def test_values_are_bf16_and_within_half_a_step():
    bits = synth.normal_bf16(71, (400, 128), 3.0)
    x = synth.bf16_bits_to_float(bits).astype(np.float64)
    codes, scales = ref.quantise(bits)
    v = ref.values(codes, scales)
    assert np.array_equal(synth.bf16_bits_to_float(synth.float_to_bf16_bits(v.astype(np.float32))), v)
    assert codes.min() >= 1 and codes.max() <= 15
    s = np.repeat(synth.bf16_bits_to_float(scales).astype(np.float64), 32, -1)
    # half a step, and what the largest channel loses where 7 s fell short of it: the
    # scale is off by at most 2^-5 of itself
    assert np.all(np.abs(v - x) <= s * (0.5 + 7 * 2.0 ** -5) + 1e-300)
    inner = np.abs(x) <= 7 * s
    assert np.all(np.abs(v - x)[inner] <= 0.5 * s[inner])


def test_special_groups():
    x = np.zeros((5, 64), np.float32)
    x[1, 3] = np.nan
    x[2, 40] = -np.inf
    x[3, :] = 3e38
    x[4, 0] = 1e-39  # a subnormal
    codes, scales = ref.quantise(synth.float_to_bf16_bits(x))
    v = ref.values(codes, scales)
    assert np.all(v[0] == 0)
    assert np.all(np.isnan(v[1, :32])) and np.all(v[1, 32:] == 0)
    assert np.all(v[2, :32] == 0) and np.all(np.isnan(v[2, 32:]))
    assert np.all(np.isfinite(v[3])) and np.allclose(v[3], 3e38, rtol=0.05)
    assert np.all(np.isfinite(v[4]))


# --------------------------------------------------------------------------- #
# gradient formula against differences
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_formula_matches_differences(interleaved, norm):
    B, T, H, D, rot = 1, 2, 2, 64, 32
    x = synth.normals(81, B * T * H * D).reshape(B, T, H, D)
    g = synth.normals(82, B * T * H * D).reshape(B, T, H, D)
    w = 1 + 0.1 * synth.normals(83, D) if norm else None
    cs = ref.table(40, rot)[np.array([[5, 39]])]
    dx, dw, _ = ref.norm_rope_bwd(g, x, w, cs, interleaved)
    h = 1e-6

    def loss(xx, ww):
        return float((ref.norm_rope(xx, ww, cs, interleaved) * g).sum())

    for i in range(0, x.size, 17):
        e = np.zeros(x.size)
        e[i] = h
        e = e.reshape(x.shape)
        d = (loss(x + e, w) - loss(x - e, w)) / (2 * h)
        assert abs(d - dx.flat[i]) <= 1e-7 * (1 + abs(d))
    if norm:
        for i in range(0, D, 7):
            e = np.zeros(D)
            e[i] = h
            d = (loss(x, w + e) - loss(x, w - e)) / (2 * h)
            assert abs(d - dw[i]) <= 1e-7 * (1 + abs(d))


# --------------------------------------------------------------------------- #
# argument checks of the C entry points
# --------------------------------------------------------------------------- #
def st(*s):
    return (ctypes.c_int64 * 3)(*s)


GOOD = dict(q=A16, k=A16, v=A16, qs=(2048, 1024, 64), ks=(2048, 1024, 64), vs=(2048, 1024, 64),
            qw=A16, kw=A16, cs=A16, pos=None, B=2, T=2, Hq=4, Hkv=2, D=64, rot=64, mp=100, il=0,
            eps=1e-6)
INV, UNS, OK = gb.ATTN_ERR_INVALID_ARG, gb.ATTN_ERR_UNSUPPORTED, gb.ATTN_OK

ROPE_BAD = [
    (dict(D=96), UNS), (dict(rot=20), UNS), (dict(rot=72), INV), (dict(rot=-8), INV),
    (dict(rot=0), INV), (dict(cs=None), INV), (dict(cs=A16 + 4), INV), (dict(mp=0), INV),
    (dict(il=2), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(qw=A16 + 2), INV), (dict(pos=A16 + 2), INV),
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(Hq=-1), INV), (dict(k=A16 + 2), INV),
    (dict(qs=(2048, 1024, 60)), INV), (dict(ks=(-2048, 1024, 64)), INV), (dict(vs=None), INV),
    (dict(B=0), OK), (dict(T=0), OK), (dict(B=1 << 20, T=1 << 15), UNS),
]


def call_fwd(kw):
    a = GOOD | dict(qo=A16, ko=A16, vo=A16) | kw
    s = {n: st(*a[n]) if a[n] else None for n in ("qs", "ks", "vs")}
    return gb.lib().qkv_norm_rope(a["q"], a["k"], a["v"], s["qs"], s["ks"], s["vs"], a["qw"],
                                  a["kw"], a["cs"], a["pos"], a["B"], a["T"], a["Hq"], a["Hkv"],
                                  a["D"], a["rot"], a["mp"], a["il"], a["eps"], a["qo"], a["ko"],
                                  a["vo"], None)


@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(q=None), INV), (dict(ko=None), INV), (dict(vo=A16 + 8), INV), (dict(Hq=0), INV),
    (dict(q=None, k=None, v=None, qo=None, ko=None, vo=None), INV),
])
def test_qkv_norm_rope_refusals(kw, code):
    assert call_fwd(kw) == code


def call_bwd(kw):
    a = GOOD | dict(gq=A16, gk=A16, gv=A16, dq=A16, dk=A16, dv=A16, ds=(2048, 1024, 64), dqw=A16,
                    dkw=A16, ws=A16, wsb=1 << 20) | kw
    s = {n: st(*a[n]) if a[n] else None for n in ("qs", "ks", "ds")}
    return gb.lib().qkv_norm_rope_bwd(a["gq"], a["gk"], a["gv"], a["q"], a["k"], s["qs"], s["ks"],
                                      a["qw"], a["kw"], a["cs"], a["pos"], a["B"], a["T"],
                                      a["Hq"], a["Hkv"], a["D"], a["rot"], a["mp"], a["il"],
                                      a["eps"], a["dq"], a["dk"], a["dv"], s["ds"], s["ds"],
                                      s["ds"], a["dqw"], a["dkw"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [x for x in ROPE_BAD if "vs" not in x[0] and x[1] != OK][:-1] + [
    (dict(B=1 << 20, T=1 << 15, ds=(1 << 25, 1024, 64)), UNS), (dict(dqw=None), INV), (dict(kw=None), INV), (dict(ws=None), INV), (dict(wsb=511), INV),
    (dict(q=None), INV), (dict(gq=None, dq=None), INV), (dict(gv=None), INV),
    (dict(dk=A16 + 2), INV),
    (dict(ds=(0, 1024, 64)), INV),      # two batches in one place
    (dict(ds=(2048, 64, 64)), INV),     # tokens over heads
    (dict(ds=(2048, 1024, 32)), INV),   # heads over channels
    (dict(B=0, qw=None, kw=None, dqw=None, dkw=None), OK),
])
def test_qkv_norm_rope_bwd_refusals(kw, code):
    assert call_bwd(kw) == code


def call_append(four, kw):
    a = GOOD | dict(pool=A16, vpool=A16, bt=A16, sl=A16, nsl=None, bs=16, mb=10, nb=30,
                    qo=A16) | kw
    s = {n: st(*a[n]) if a[n] else None for n in ("qs", "ks", "vs")}
    pools = (a["pool"],) if four else (a["pool"], a["vpool"])
    f = gb.lib().paged_kv4_append if four else gb.lib().paged_qkv_append
    return f(a["q"], a["k"], a["v"], s["qs"], s["ks"], s["vs"], a["qw"], a["kw"], a["cs"],
             a["pos"], *pools, a["bt"], a["sl"], a["nsl"], a["bs"], a["B"], a["T"], a["Hq"],
             a["Hkv"], a["D"], a["mb"], a["nb"], a["rot"], a["mp"], a["il"], a["eps"], a["qo"],
             None)


@pytest.mark.parametrize("sizes", [
    dict(B=1, T=1, Hq=1 << 30, Hkv=1 << 30),        # heads past an int
    dict(B=1, T=1, Hq=(1 << 31) - 1, Hkv=1),
    dict(B=1, T=300, Hq=1 << 24, Hkv=1),            # 2^32 rows and more
    dict(B=50, T=50, Hq=64, Hkv=1 << 20),
])
def test_more_rows_than_a_launch_counts_are_refused(sizes):
    """As a size that is not supported, not as a CUDA error and not as a call that does nothing."""
    strides = dict(qs=(0, 0, 64), ks=(0, 0, 64), vs=(0, 0, 64))
    assert call_fwd(sizes | strides) == UNS
    assert call_append(False, sizes | strides) == UNS and call_append(True, sizes | strides) == UNS
    rows = max(sizes["Hq"], sizes["Hkv"]) * 64
    places = (rows * sizes["T"], rows, 64)
    assert call_bwd(sizes | strides | dict(ds=places)) == UNS


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(bs=8), UNS), (dict(mb=0), INV), (dict(nb=0), INV), (dict(Hkv=0), INV),
    (dict(pool=None), INV), (dict(pool=A16 + 8), INV), (dict(bt=None), INV), (dict(sl=None), INV),
    (dict(sl=A16 + 2), INV), (dict(nsl=A16 + 4), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(q=None), INV), (dict(qo=None), INV), (dict(nb=1 << 28), UNS), (dict(mb=1 << 28), UNS),
    (dict(T=0, nsl=A16 + 4), INV), (dict(T=0, nsl=A16, sl=None), INV), (dict(B=0, nsl=A16), OK),
])
def test_append_refusals(four, kw, code):
    assert call_append(four, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(bs=32), UNS), (dict(D=32), UNS), (dict(S=-1), INV), (dict(ml=-1), INV),
    (dict(pool=None), INV), (dict(pool=A16 + 4), INV), (dict(ko=None), INV), (dict(vo=A16 + 2), INV),
    (dict(sl=None), INV), (dict(S=0), OK), (dict(ml=0), OK), (dict(S=1 << 30, ml=64), UNS),
])
def test_kv4_gather_refusals(kw, code):
    a = dict(pool=A16, bt=A16, sl=A16, bs=16, S=2, Hkv=2, D=64, mb=4, nb=9, ml=64, ko=A16,
             vo=A16) | kw
    assert gb.lib().paged_kv4_gather(a["pool"], a["bt"], a["sl"], a["bs"], a["S"], a["Hkv"],
                                     a["D"], a["mb"], a["nb"], a["ml"], a["ko"], a["vo"],
                                     None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(bs=8), UNS), (dict(D=96), UNS), (dict(Hq=34), UNS), (dict(Hq=5), INV), (dict(Hkv=0), INV),
    (dict(q=None), INV), (dict(pool=None), INV), (dict(pool=A16 + 8), INV), (dict(o=None), INV),
    (dict(bt=None), INV), (dict(sl=A16 + 2), INV), (dict(lse=A16 + 1), INV), (dict(ws=None), INV),
    (dict(ws=A16 + 16), INV), (dict(wsb=-1), INV), (dict(scale=0.0), INV),
    (dict(scale=float("nan")), INV), (dict(msl=-1), INV), (dict(mb=0), INV), (dict(nb=0), INV),
    (dict(nb=1 << 27), UNS), (dict(mb=1 << 28), UNS), (dict(S=-1), INV), (dict(S=0), OK),
])
def test_kv4_decode_refusals(kw, code):
    a = dict(q=A16, pool=A16, bt=A16, sl=A16, bs=16, S=4, Hq=12, Hkv=2, D=128, mb=512, nb=1000,
             msl=8192, scale=0.088, o=A16, lse=None, ws=A16, wsb=0) | kw
    need = gb.paged_kv4_attn_decode_workspace_size(a["S"], a["Hq"], a["Hkv"], a["D"], a["msl"])
    assert gb.lib().paged_kv4_attn_decode(a["q"], a["pool"], a["bt"], a["sl"], a["bs"], a["S"],
                                          a["Hq"], a["Hkv"], a["D"], a["mb"], a["nb"], a["msl"],
                                          a["scale"], a["o"], a["lse"], a["ws"],
                                          max(0, need + a["wsb"]), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(bs=8), UNS), (dict(D=96), UNS), (dict(Hq=5), INV), (dict(Hkv=0), INV), (dict(Tq=-1), INV),
    (dict(q=None), INV), (dict(q=A16 + 8), INV), (dict(pool=None), INV), (dict(pool=A16 + 8), INV),
    (dict(o=None), INV), (dict(bt=None), INV), (dict(sl=A16 + 2), INV), (dict(lse=A16 + 1), INV),
    (dict(causal=2), INV), (dict(scale=-1.0), INV), (dict(scale=float("inf")), INV),
    (dict(ml=-1), INV), (dict(mb=0), INV), (dict(nb=0), INV), (dict(nb=1 << 27), UNS),
    (dict(mb=1 << 28), UNS), (dict(B=0), OK), (dict(Tq=0), OK), (dict(ws=None), INV),
    (dict(ws=A16 + 16), INV), (dict(wsb=-1), INV),
])
def test_kv4_prefill_refusals(kw, code):
    a = dict(q=A16, pool=A16, bt=A16, sl=A16, bs=16, B=4, Hq=12, Hkv=2, Tq=9, D=128, mb=512,
             nb=1000, ml=8192, causal=1, scale=0.088, o=A16, lse=None, ws=A16, wsb=0) | kw
    need = gb.paged_kv4_attn_prefill_workspace_size(a["B"], a["Hq"], a["Hkv"], a["Tq"], a["D"],
                                                    a["ml"])
    assert gb.lib().paged_kv4_attn_prefill(a["q"], a["pool"], a["bt"], a["sl"], a["bs"], a["B"],
                                           a["Hq"], a["Hkv"], a["Tq"], a["D"], a["mb"], a["nb"],
                                           a["ml"], a["causal"], a["scale"], a["o"], a["lse"],
                                           a["ws"], max(0, need + a["wsb"]), None) == code


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,Hkv,B", [(17, 1, 1), (17, 2, 9), (24, 1, 1), (32, 1, 8), (40, 3, 2)])
def test_single_tokens_of_wide_groups_have_a_workspace(group, Hkv, B, D):
    """More query heads on a KV head than one pass takes (16) are several segments, whose
    results meet in the workspace: one-launch decoding, a CTA a KV head, is not for them."""
    size = gb.paged_kv4_attn_prefill_workspace_size
    for ml in (513, 1024, 1025, 100000):
        assert size(B, group * Hkv, Hkv, 1, D, ml) > 0
    if B * group * Hkv > 152:  # (fewer units on so short a cache: tiles)
        assert size(B, group * Hkv, Hkv, 1, D, 512) > 0
    assert size(B, 16 * Hkv, Hkv, 1, D, 1024) == 0


def test_chunks_past_the_row_kernels_counts_are_the_tile_kernels():
    """A length bound that makes 2^31 steps of 64 tokens or more: no rows, so no workspace."""
    size, top = gb.paged_kv4_attn_prefill_workspace_size, 2 ** 31 - 1
    assert size(31, 4, 2, 4, 128, top) > 0
    assert size(32, 4, 2, 4, 128, top) == 0
    assert size(1 << 20, 4, 2, 1, 128, 1 << 20) == 0


def test_workspace_sizes_at_the_largest_length_bound():
    """At 2^31 - 1 tokens a batch has its most ranges (2048), and a piece more a segment."""
    for ml in (2 ** 31 - 1, 2 ** 31 - 64, 1 << 20):
        pieces = 2048 + 3 * 2
        n = pieces * 2 * (128 + 1) * 4
        need = gb.paged_kv4_attn_decode_workspace_size(3, 4, 2, 128, ml)
        assert n <= need <= n + 2 * 4 * 6 + 4 * 256


# --------------------------------------------------------------------------- #
# argument checks of the binding
# --------------------------------------------------------------------------- #
torch = pytest.importorskip("torch")


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


@pytest.mark.parametrize("bad", [
    dict(q=bf(2, 3, 4, 32)), dict(q=bf(2, 3, 4, 64).float()), dict(k=bf(2, 4, 2, 64)),
    dict(v=bf(2, 3, 3, 64)), dict(q=bf(2, 3, 4, 128)[..., ::2]), dict(cos_sin=torch.zeros(9)),
    dict(cos_sin=torch.zeros(9, 64, dtype=torch.float64)), dict(q_weight=torch.ones(64)),
    dict(k_weight=bf(32)), dict(positions=torch.zeros(2, 3)),
    dict(positions=torch.zeros(3, 2, dtype=torch.int32)), dict(q_out=bf(2, 3, 4, 64)),
    dict(v=None, v_out=bf(2, 2, 3, 64)), dict(q=None, k=None, v=None), {},
])
def test_binding_refuses_bad_rope_operands(bad):
    a = dict(q=bf(2, 3, 4, 64), k=bf(2, 3, 2, 64), v=bf(2, 3, 2, 64), cos_sin=torch.zeros(9, 64))
    with pytest.raises(ValueError):  # with nothing bad: the tensors are not on a GPU
        gb.qkv_norm_rope(**(a | bad))


ROPE = dict(q=(2, 3, 4, 64), k=(2, 3, 2, 64), v=(2, 3, 2, 64), cos_sin=(9, 64), q_weight=(64,),
            k_weight=(64,))
GRADS = dict(dq_out=(2, 4, 3, 64), dk_out=(2, 2, 3, 64), dv_out=(2, 2, 3, 64)) | {
    n: ROPE[n] for n in ("q", "k", "cos_sin", "q_weight", "k_weight")}
DIFFERENTIABLE = [(gb.qkv_norm_rope, ROPE, n) for n in ROPE] + [
    (gb.qkv_norm_rope_bwd, GRADS, n) for n in GRADS]


@pytest.mark.parametrize("op,shapes,name", DIFFERENTIABLE, ids=lambda x: getattr(x, "__name__", None) or str(x)[:9])
def test_operands_of_automatic_differentiation_are_refused(op, shapes, name):
    """Outputs have no way back to their operands, so a call that would lose a gradient
    without a word is refused, in reverse and in forward mode."""
    a = {n: torch.zeros(s, dtype=torch.float32 if n == "cos_sin" else torch.bfloat16)
         for n, s in shapes.items()}
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(a[name], torch.ones_like(a[name]))
        with pytest.raises(ValueError, match=f"{op.__name__} records nothing.*and {name} takes"):
            op(**a | {name: dual})
    a[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{op.__name__} records nothing.*and {name} takes"):
        op(**a)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # as without a gradient
        op(**a)


@pytest.mark.parametrize("bad", [
    dict(dk_out=bf(2, 2, 4, 64)), dict(q=None), dict(q=bf(2, 3, 5, 64)), dict(dq=bf(2, 4, 3, 64)),
    dict(dq_weight=bf(64)), dict(k_weight=None, dk_weight=torch.zeros(64)),
    dict(dv_out=None, dv=bf(2, 3, 2, 64)), dict(workspace=torch.zeros(8)), {},
])
def test_binding_refuses_bad_gradients(bad):
    a = dict(dq_out=bf(2, 4, 3, 64), dk_out=bf(2, 2, 3, 64), dv_out=bf(2, 2, 3, 64),
             q=bf(2, 3, 4, 64), k=bf(2, 3, 2, 64), q_weight=bf(64), k_weight=bf(64),
             cos_sin=torch.zeros(9, 64))
    with pytest.raises(ValueError):
        gb.qkv_norm_rope_bwd(**(a | bad))


@pytest.mark.parametrize("bad", [
    dict(kv_pool=torch.zeros(9, 2, 18 * 32, dtype=torch.uint8)), dict(kv_pool=bf(9, 2, 18 * 64)),
    dict(kv_pool=torch.zeros(9, 2, 16, 64, dtype=torch.uint8)),
    dict(seq_lens=torch.zeros(3, dtype=torch.int32)), dict(seq_lens=torch.zeros(2)),
    dict(block_table=torch.zeros(3, 4, dtype=torch.int32)), dict(q_out=bf(2, 4, 3, 64)),
    dict(q=None, q_out=bf(2, 4, 1, 64)), dict(new_seq_lens=torch.zeros(3, dtype=torch.int32)), {},
])
def test_binding_refuses_bad_appends(bad):
    a = dict(q=bf(2, 1, 4, 64), k=bf(2, 1, 2, 64), v=bf(2, 1, 2, 64),
             kv_pool=torch.zeros(9, 2, 18 * 64, dtype=torch.uint8),
             block_table=torch.zeros(2, 4, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gb.paged_kv4_append(**(a | bad))


@pytest.mark.parametrize("bad", [
    dict(kv_pool=torch.zeros(9, 2, 18 * 32, dtype=torch.uint8)), dict(kv_pool=bf(9, 2, 16, 64)),
    dict(kv_pool=torch.zeros(9, 2, 100, dtype=torch.uint8)), dict(q=torch.zeros(2, 4, 64)),
    dict(out=bf(2, 5, 64)), dict(lse=bf(2, 4)), dict(block_table=torch.zeros(2, 4)),
    dict(seq_lens=torch.zeros(3, dtype=torch.int32)), {},
])
def test_binding_refuses_bad_kv4_attention(bad):
    a = dict(q=bf(2, 4, 64), kv_pool=torch.zeros(9, 2, 18 * 64, dtype=torch.uint8),
             block_table=torch.zeros(2, 4, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), max_seq_len=64)
    with pytest.raises(ValueError):
        gb.paged_kv4_attn_decode(**(a | bad))
    a |= bad
    a["kv_lens"], a["max_kv_len"] = a.pop("seq_lens"), a.pop("max_seq_len")
    a = {n: t.unsqueeze(2) if n in ("q", "out", "lse") else t for n, t in a.items()}
    with pytest.raises(ValueError):
        gb.paged_kv4_attn_prefill(**a)


def test_tables_past_an_int_are_refused():
    """Sizes that the C ABI's ints would wrap (on the meta device: nothing is allocated)."""
    def meta(*s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device="meta")

    i32, u8, wide = torch.int32, torch.uint8, (1 << 32) + 4
    rows = dict(q=meta(2, 1, 4, 64), k=meta(2, 1, 2, 64), v=meta(2, 1, 2, 64))
    table, lens, pool = meta(2, wide, dtype=i32), meta(2, dtype=i32), meta(9, 2, 18 * 64, dtype=u8)
    with pytest.raises(ValueError, match="cos_sin"):
        gb.qkv_norm_rope(**rows, cos_sin=meta(wide, 64, dtype=torch.float32))
    calls = [
        lambda: gb.paged_kv4_append(**rows, kv_pool=pool, block_table=table, seq_lens=lens),
        lambda: gb.paged_qkv_append(**rows, k_pool=meta(9, 2, 16, 64), v_pool=meta(9, 2, 16, 64),
                                    block_table=table, seq_lens=lens),
        lambda: gb.paged_kv4_gather(pool, table, lens, 64),
        lambda: gb.paged_kv4_attn_decode(meta(2, 4, 64), pool, table, lens, 64),
        lambda: gb.paged_kv4_attn_prefill(meta(2, 4, 1, 64), pool, table, lens, 64),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="block_table"):
            call()


def test_first_calls_of_two_threads(monkeypatch):
    """A call that another thread makes at any point of the first one's loading of torch finds
    all of what it uses (each line of the loader is such a point)."""
    import sys
    import threading

    a = dict(q=bf(2, 3, 4, 64), k=bf(2, 3, 2, 64), v=bf(2, 3, 2, 64), cos_sin=torch.zeros(9, 64))
    gb.lib()

    def refusal():  # with all in place: the tensors are not on a GPU
        try:
            gb.qkv_norm_rope(**a)
        except Exception as e:  # noqa: BLE001 -- whatever a half-loaded state leads to
            seen.append(repr(e))

    def trace(frame, event, arg):
        if frame.f_code is gb._load_torch.__code__ and event != "return":
            if events[0] == point:
                t = threading.Thread(target=refusal)
                t.start()
                t.join(60)
            events[0] += 1
            return trace

    point, last = 0, 1
    while point < last:
        for n in ("_torch", "_Tensor", "_bf16", "_f32", "_i32", "_u8", "_quick"):
            monkeypatch.setattr(gb, n, None)
        seen, events, before = [], [0], sys.gettrace()
        sys.settrace(trace)
        try:
            refusal()
        finally:
            sys.settrace(before)
        assert len(seen) == 2 and all("ValueError" in s and "CUDA" in s for s in seen), (point, seen)
        point, last = point + 1, events[0]
    assert last > 4
