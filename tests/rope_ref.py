"""References for the norm + rotation pass and the 4-bit cache (test infrastructure
only): float64 numpy from the definitions, on bf16 bit patterns (uint16) or float64."""

from __future__ import annotations

import numpy as np

import synth

EPS = 1e-6
BS = 16


def table(max_pos, rot, theta=1e4):
    """[max_pos, rot] float32: cosines, then sines."""
    inv = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(max_pos, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def planes(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope(x, w, cs, interleaved, eps=EPS):
    """x [B, T, H, D] float64, w [D] or None, cs [B, T, rot] rows of the table or None."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    if cs is not None:
        rot = cs.shape[-1]
        a, b = planes(rot, interleaved)
        c, s = cs[:, :, None, :rot // 2].astype(np.float64), cs[:, :, None, rot // 2:].astype(np.float64)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a] = ya * c - yb * s
        y[..., b] = yb * c + ya * s
    return y


def norm_rope_bwd(g, x, w, cs, interleaved, eps=EPS):
    """Gradient g [B, T, H, D] of the output -> (dx, dw, sum of |terms| of dw)."""
    u = np.array(g, dtype=np.float64)
    if cs is not None:
        rot = cs.shape[-1]
        a, b = planes(rot, interleaved)
        c, s = cs[:, :, None, :rot // 2].astype(np.float64), cs[:, :, None, rot // 2:].astype(np.float64)
        ga, gb = u[..., a].copy(), u[..., b].copy()
        u[..., a] = ga * c + gb * s
        u[..., b] = gb * c - ga * s
    if w is None:
        return u, None, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    terms = u * xh
    uw = u * w
    dx = r * (uw - xh * (uw * xh).mean(-1, keepdims=True))
    return dx, terms.sum((0, 1, 2)), np.abs(terms).sum((0, 1, 2))


def quantise(bits):
    """bf16 bits [..., D] -> (codes n + 8 uint8 [..., D], scales bf16 bits [..., D / 32]).
    Quotients of a bf16 by 7 or by a 5-bit scale are never so near a rounding border
    that float64 and float32 could round differently, so codes must match bit for bit."""
    x = synth.bf16_bits_to_float(bits).astype(np.float64)
    g = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)  # NaN propagates
        t = (amax / 7.0).astype(np.float32)
        b = t.view(np.uint32)
        b = (b + np.uint32(0x3FFFF) + ((b >> np.uint32(19)) & np.uint32(1))) & np.uint32(0xFFF80000)
        s = np.where(np.isfinite(amax), b, np.uint32(0x7FC00000)).astype(np.uint32)
        sf = s.view(np.float32).astype(np.float64)[..., None]
        n = np.where(sf > 0, np.clip(np.rint(g / np.where(sf > 0, sf, 1.0)), -7, 7), 0.0)
    return (n + 8).astype(np.uint8).reshape(x.shape), (s >> np.uint32(16)).astype(np.uint16)


def values(codes, scales):
    """float64 values that codes and scales stand for."""
    n = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, 32) - 8
    s = synth.bf16_bits_to_float(scales).astype(np.float64)
    return (n * s[..., None]).reshape(codes.shape)


def nibble(c, D, per):
    """Position of channel c in a row (per = 8 for K rows, 4 for V rows)."""
    return (c % 32 // per * (D // 32) + c // 32) * per + c % per


def pack_rows(codes, per):
    D = codes.shape[-1]
    nib = np.zeros(codes.shape, np.uint8)
    nib[..., [nibble(c, D, per) for c in range(D)]] = codes
    return nib[..., 0::2] | (nib[..., 1::2] << 4)


def write_pool(pool, block, slot, head, k_bits, v_bits):
    """One token of one KV head into pool [NB, Hkv, 18 D] uint8."""
    D = k_bits.shape[-1]
    for off, bits, per in ((0, k_bits, 8), (9 * D, v_bits, 4)):
        codes, scales = quantise(bits)
        chunk = pool[block, head]
        chunk[off + slot * D // 2:off + (slot + 1) * D // 2] = pack_rows(codes, per)
        at = off + 8 * D + slot * D // 16
        chunk[at:at + D // 16] = scales.view(np.uint8)


def pool_from_bf16(k_pool, v_pool, fill=None):
    """The 4-bit form of bf16 pools [NB, Hkv, 16, D] (bits)."""
    NB, Hkv, bs, D = k_pool.shape
    parts = []
    for bits, per in ((k_pool, 8), (v_pool, 4)):
        codes, scales = quantise(bits)
        parts.append(pack_rows(codes, per).reshape(NB, Hkv, 8 * D))
        parts.append(np.ascontiguousarray(scales).view(np.uint8).reshape(NB, Hkv, D))
    return np.concatenate(parts, 2)


def value_bits(bits):
    """bf16 bits of the values that rows of bf16 bits become in the cache (exact)."""
    v = values(*quantise(bits))
    out = synth.float_to_bf16_bits(v.astype(np.float32))
    finite = np.isfinite(v)
    assert np.array_equal(synth.bf16_bits_to_float(out)[finite].astype(np.float64), v[finite])
    return out
