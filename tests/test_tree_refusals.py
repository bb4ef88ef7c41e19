"""What the operators for trees of drafted tokens refuse before anything is launched, in the C
entry points and in the Python binding.  No GPU is needed."""

from __future__ import annotations

import ctypes

import pytest

import attention_flashattention_fwd_03_gb300 as gb

torch = pytest.importorskip("torch")

A16 = 0x100000  # a 16-byte aligned address that is never dereferenced by validation
INVALID, UNSUPPORTED, OK = gb.ATTN_ERR_INVALID_ARG, gb.ATTN_ERR_UNSUPPORTED, gb.ATTN_OK
NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the path without a device")


@pytest.fixture(scope="module")
def lib():
    return gb.lib()


def attend(lib, q=A16, k=A16, v=A16, bt=A16, sl=A16, pa=A16, tl=None, bs=16, S=4, Tn=8, Hq=12,
           Hkv=2, D=128, mb=512, nb=1000, msl=8192, scale=0.088, o=A16, lse=None, ws=A16, wsb=None):
    if wsb is None:
        wsb = 1 << 40
    return lib.paged_attn_tree(q, k, v, bt, sl, pa, tl, bs, S, Tn, Hq, Hkv, D, mb, nb, msl, scale,
                               o, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bs=8), UNSUPPORTED), (dict(D=80), UNSUPPORTED), (dict(Tn=257), UNSUPPORTED),
    (dict(Hq=258, Hkv=2), UNSUPPORTED),  # 129 query heads on a KV head
    (dict(Hq=12, Hkv=5), INVALID), (dict(Hkv=0), INVALID), (dict(S=-1), INVALID),
    (dict(Tn=-1), INVALID), (dict(mb=0), INVALID), (dict(nb=0), INVALID), (dict(msl=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(pa=None), INVALID),
    (dict(o=None), INVALID), (dict(q=A16 + 8), INVALID), (dict(k=A16 + 8), INVALID),
    (dict(v=A16 + 8), INVALID), (dict(o=A16 + 8), INVALID), (dict(bt=A16 + 2), INVALID),
    (dict(sl=A16 + 2), INVALID), (dict(pa=A16 + 2), INVALID), (dict(tl=A16 + 2), INVALID),
    (dict(lse=A16 + 2), INVALID),
    (dict(nb=1 << 27), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(S=1 << 20, Hq=512, Hkv=2), UNSUPPORTED),
    (dict(S=1 << 24, Hq=2, Hkv=2, Tn=1, msl=2 ** 31 - 1), UNSUPPORTED),
    (dict(S=0, q=None, o=None), OK), (dict(Tn=0, q=None, o=None), OK),
])
def test_attention(lib, kw, code):
    assert attend(lib, **kw) == code


def test_attention_workspace(lib):
    size = lib.paged_attn_tree_workspace_size
    assert size(-1, 8, 12, 2, 128, 8192) == 0 and size(4, 0, 12, 2, 128, 8192) == 0
    assert size(4, 257, 12, 2, 128, 8192) == 0 and size(4, 8, 12, 5, 128, 8192) == 0
    assert size(4, 8, 258, 2, 128, 8192) == 0
    assert size(4, 8, 12, 2, 96, 8192) == 0 and size(1 << 30, 256, 64, 2, 128, 2 ** 31 - 1) == 0
    for S, Tn, Hq, Hkv, D, msl in [(1, 1, 1, 1, 64, 1), (64, 8, 12, 2, 128, 8200), (3, 256, 64, 4, 64, 5000),
                                   (1, 4, 8, 8, 128, 2 ** 31 - 1), (5000, 2, 2, 1, 64, 70000)]:
        need = size(S, Tn, Hq, Hkv, D, msl)
        kw = dict(S=S, Tn=Tn, Hq=Hq, Hkv=Hkv, D=D, msl=msl)
        # a piece a CTA range and its successor, D + 1 words of every row of a unit
        assert 0 <= need <= 2 * 160 * 256 * (D + 1) * 4 + (1 << 16)
        if need:
            assert attend(lib, wsb=need - 1, **kw) == INVALID
            assert attend(lib, ws=None, **kw) == INVALID
            assert attend(lib, ws=A16 + 16, **kw) == INVALID


def verify(lib, p=A16, q=A16, ps=(800, 100), qs=(800, 100), kind=0, tok=A16, pa=A16, u=A16,
           tl=None, S=4, Tn=8, V=100, out=A16, path=A16, counts=A16):
    arr = lambda s: None if s is None else (ctypes.c_int64 * 3)(*s)  # noqa: E731
    return lib.draft_verify(p, q, arr(ps), arr(qs), kind, tok, pa, u, tl, S, Tn, V, out, path, counts,
                            None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(Tn=-1), INVALID), (dict(V=0), INVALID), (dict(V=-5), INVALID),
    (dict(kind=2), INVALID), (dict(kind=-1), INVALID), (dict(Tn=257), UNSUPPORTED),
    (dict(V=1 << 30), UNSUPPORTED), (dict(S=1 << 26), UNSUPPORTED),
    (dict(p=None), INVALID), (dict(tok=None), INVALID), (dict(pa=None), INVALID),
    (dict(u=None), INVALID), (dict(out=None), INVALID), (dict(path=None), INVALID),
    (dict(counts=None), INVALID), (dict(ps=None), INVALID), (dict(qs=None), INVALID),
    (dict(ps=(-1, 100)), INVALID), (dict(qs=(800, -1)), INVALID), (dict(ps=(1 << 50, 0)), INVALID),
    (dict(p=A16 + 2), INVALID), (dict(q=A16 + 2), INVALID), (dict(p=A16 + 1, kind=1), INVALID),
    (dict(tok=A16 + 2), INVALID), (dict(pa=A16 + 2), INVALID), (dict(u=A16 + 2), INVALID),
    (dict(tl=A16 + 2), INVALID), (dict(out=A16 + 2), INVALID), (dict(path=A16 + 1), INVALID),
    (dict(counts=A16 + 2), INVALID), (dict(S=0, p=None), OK),
])
def test_verify(lib, kw, code):
    assert verify(lib, **kw) == code


def keep(lib, layers=2, k=None, v=None, bt=A16, sl=A16 + (1 << 16), path=A16 + (2 << 16),
         counts=A16 + (3 << 16), new=A16 + (4 << 16), bs=16, S=4, n=8, Hkv=2, D=128, mb=10, nb=100,
         null=False):
    arr = lambda x, at: (ctypes.c_void_p * max(layers, 1))(  # noqa: E731
        *(x or [(at << 40) + (i << 20) for i in range(max(layers, 1))]))
    return lib.paged_kv_keep(None if null else arr(k, 1), arr(v, 2), layers, bt, sl, path, counts, new, bs,
                             S, n, Hkv, D, mb, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(layers=0), INVALID), (dict(layers=-1), INVALID), (dict(S=-1), INVALID),
    (dict(n=-1), INVALID), (dict(Hkv=0), INVALID), (dict(mb=0), INVALID), (dict(nb=0), INVALID),
    (dict(bs=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(n=257), UNSUPPORTED),
    (dict(nb=1 << 27), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(null=True), INVALID), (dict(k=[A16, None]), INVALID), (dict(v=[None, A16]), INVALID),
    (dict(k=[A16, A16 + 8]), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID),
    (dict(path=None), INVALID), (dict(counts=None), INVALID), (dict(bt=A16 + 2), INVALID),
    (dict(sl=A16 + 2), INVALID), (dict(path=A16 + 2), INVALID), (dict(counts=A16 + 2), INVALID),
    (dict(new=A16 + 2), INVALID),
    (dict(new=A16 + (1 << 16)), INVALID), (dict(new=A16 + (1 << 16) + 12), INVALID),
    (dict(new=A16 + (2 << 16) + 124), INVALID), (dict(new=A16 + (3 << 16) - 12), INVALID),
    (dict(new=A16 + 156), INVALID), (dict(S=0, bt=None), OK),
])
def test_keep(lib, kw, code):
    assert keep(lib, **kw) == code


@NO_DEVICE
def test_valid_calls_without_a_device_are_errors(lib):
    assert attend(lib) == gb.ATTN_ERR_CUDA
    assert verify(lib) == gb.ATTN_ERR_CUDA and verify(lib, q=None, qs=None) == gb.ATTN_ERR_CUDA
    assert verify(lib, kind=1, p=A16 + 2) == gb.ATTN_ERR_CUDA
    assert verify(lib, Tn=0, p=None, tok=None, pa=None, u=None, out=None, path=None) == gb.ATTN_ERR_CUDA
    assert keep(lib) == gb.ATTN_ERR_CUDA and keep(lib, new=None) == gb.ATTN_ERR_CUDA
    assert keep(lib, n=0, path=None) == gb.ATTN_ERR_CUDA


@NO_DEVICE
def test_pools_that_share_memory(lib):
    """A pool of nb 100, Hkv 2, D 128 has 819200 bytes."""
    at, pool = 1 << 40, 819200
    k, v = [at + i * pool for i in range(3)], [at + (3 + i) * pool for i in range(3)]
    for x, y in ((k, v), (v, k), (k[::-1], v), (k, v[::-1]), (k[::2] + v[1:2], v[::2] + k[1:2])):
        assert keep(lib, layers=3, k=x, v=y) == gb.ATTN_ERR_CUDA
    paired = [at + 2 * i * pool for i in range(3)]
    assert keep(lib, layers=3, k=paired, v=[x + pool for x in paired]) == gb.ATTN_ERR_CUDA
    assert keep(lib, layers=1, k=k[:1], v=k[1:2]) == gb.ATTN_ERR_CUDA
    many = [at + i * pool for i in range(600)]
    assert keep(lib, layers=300, k=many[::2], v=many[1::2]) == gb.ATTN_ERR_CUDA
    assert keep(lib, layers=300, k=many[::2], v=many[1::2][:-1] + many[:1]) == INVALID
    for x, y in ((k, k), ([k[0], k[0], k[2]], v), (k, [v[0], v[1], v[0]]), (k, v[:2] + k[2:]),
                 (k, [v[0] - 16, v[1], v[2]]), ([k[0], k[1], k[2] + 16], v),
                 ([k[0], k[0] + pool - 16, k[2]], v)):
        assert keep(lib, layers=3, k=x, v=y) == INVALID
    assert keep(lib, layers=1, k=k[:1], v=k[:1]) == INVALID


def test_long_bounds_on_many_requests(lib):
    """What the counts hold: segments x (key tiles + 2) x 20 below 2^31."""
    size = lib.paged_attn_tree_workspace_size
    assert size(4000, 8, 32, 8, 128, 400000) > 0 and size(1000, 200, 64, 8, 128, 1 << 20) > 0
    tiles = (2 ** 31 - 1) // (20 * 32000) - 2
    assert size(4000, 8, 32, 8, 128, 128 * tiles) > 0
    assert size(4000, 8, 32, 8, 128, 128 * tiles + 1) == 0
    assert attend(lib, S=4000, Tn=8, Hq=32, Hkv=8, msl=128 * tiles + 1) == UNSUPPORTED


# --------------------------------------------------------------------------- #
# the Python binding: metadata only, so CPU tensors reach the check that fails first
# --------------------------------------------------------------------------- #
def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def attend_args():
    return dict(q=bf16(2, 4, 3, 64), k_pool=bf16(9, 2, 16, 64), v_pool=bf16(9, 2, 16, 64),
                block_table=i32(2, 5), seq_lens=i32(2), parents=i32(2, 3), max_seq_len=80)


@pytest.mark.parametrize("change,match", [
    (dict(q=bf16(2, 4, 64)), "4-d"), (dict(q=bf16(2, 4, 3, 64).float()), "q must be"),
    (dict(q=bf16(2, 3, 4, 64).transpose(1, 2)), "q must be contiguous"),
    (dict(k_pool=bf16(9, 2, 16, 128), v_pool=bf16(9, 2, 16, 128)), "inconsistent"),
    (dict(v_pool=bf16(8, 2, 16, 64)), "v_pool"), (dict(k_pool=bf16(2, 16, 64)), "k_pool"),
    (dict(block_table=i32(3, 5)), "block_table"), (dict(block_table=i32(2, 5).long()), "block_table"),
    (dict(seq_lens=i32(3)), "seq_lens"), (dict(parents=i32(2, 4)), "parents"),
    (dict(parents=i32(2, 3).long()), "parents"), (dict(tree_lens=i32(3)), "tree_lens"),
    (dict(tree_lens=i32(2).long()), "tree_lens"), (dict(out=bf16(2, 4, 3, 128)), "out"),
    (dict(lse=torch.zeros(2, 4, 4)), "lse"), (dict(workspace=i32(9)), "workspace"),
    (dict(max_seq_len=-1), "length"), (dict(max_seq_len=1 << 31), "length"),
    (dict(), "CUDA tensors"),
])
def test_attention_binding(change, match):
    with pytest.raises(ValueError, match=match):
        gb.paged_attn_tree(**{**attend_args(), **change})
    with pytest.raises(TypeError):
        gb.paged_attn_tree(**{**attend_args(), "q": 3})


def verify_args():
    return dict(target_probs=torch.zeros(2, 3, 10), draft_probs=torch.zeros(2, 3, 10),
                draft_tokens=i32(2, 3), parents=i32(2, 3), uniforms=torch.zeros(2, 3))


@pytest.mark.parametrize("change,match", [
    (dict(target_probs=torch.zeros(2, 30)), "target_probs"),
    (dict(target_probs=torch.zeros(2, 3, 10).double()), "target_probs"),
    (dict(target_probs=torch.zeros(2, 3, 10).half()), "target_probs"),
    (dict(target_probs=torch.zeros(2, 10, 3).transpose(1, 2)), "contiguous rows"),
    (dict(draft_probs=torch.zeros(2, 3, 11)), "draft_probs"),
    (dict(draft_probs=bf16(2, 3, 10)), "draft_probs"),
    (dict(draft_probs=torch.zeros(2, 10, 3).transpose(1, 2)), "contiguous rows"),
    (dict(draft_tokens=i32(2, 4)), "draft_tokens"), (dict(draft_tokens=i32(2, 3).long()), "draft_tokens"),
    (dict(parents=i32(3, 2)), "parents"), (dict(uniforms=torch.zeros(2, 3).double()), "uniforms"),
    (dict(tree_lens=i32(2, 1)), "tree_lens"), (dict(tokens_out=i32(2, 4)), "tokens_out"),
    (dict(path=i32(2, 3).long()), "path"), (dict(counts=i32(3)), "counts"), (dict(), "CUDA tensors"),
])
def test_verify_binding(change, match):
    with pytest.raises(ValueError, match=match):
        gb.draft_verify(**{**verify_args(), **change})


def keep_args():
    return dict(k_pool=bf16(9, 2, 16, 64), v_pool=bf16(9, 2, 16, 64), block_table=i32(2, 5),
                seq_lens=i32(2), path=i32(2, 3), counts=i32(2))


@pytest.mark.parametrize("change,match", [
    (dict(v_pool=bf16(8, 2, 16, 64)), "same layers"), (dict(v_pool=[bf16(9, 2, 16, 64)] * 2), "same layers"),
    (dict(k_pool=[bf16(9, 2, 16, 64), bf16(8, 2, 16, 64)]), "one shape"),
    (dict(k_pool=bf16(9, 2, 16, 64).float()), "k_pool"), (dict(k_pool=bf16(2, 16, 64)), "k_pool"),
    (dict(k_pool=bf16(2, 9, 2, 16, 128)[..., :64]), "k_pool must be contiguous"),
    (dict(k_pool=[], v_pool=[]), "one layer"), (dict(seq_lens=i32(2, 1)), "1-d"),
    (dict(block_table=i32(3, 5)), "block_table"), (dict(path=i32(6)), "path"),
    (dict(path=i32(3, 3)), "path"), (dict(path=i32(2, 3).long()), "path"),
    (dict(counts=i32(3)), "counts"), (dict(new_seq_lens=i32(3)), "new_seq_lens"), (dict(), "CUDA tensors"),
])
def test_keep_binding(change, match):
    with pytest.raises(ValueError, match=match):
        gb.paged_kv_keep(**{**keep_args(), **change})


def test_sizes_past_the_c_abi_are_refused():
    """Sizes that a C int would wrap (tensors without memory)."""
    a = {k: v.to("meta") for k, v in verify_args().items()}
    p = torch.empty(2, 3, 1 << 31, device="meta")
    with pytest.raises(ValueError, match="V = "):
        gb.draft_verify(**{**a, "target_probs": p, "draft_probs": None})
    a = {k: v.to("meta") for k, v in keep_args().items()}
    pool = torch.empty(1 << 31, 2, 16, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="NB = "):
        gb.paged_kv_keep(**{**a, "k_pool": pool, "v_pool": pool})
