"""The operators between a model's QKV projection and its attention output: cases,
their plain form in elementary torch operations, and the library's calls.

Kinds of cases:

  rope, rope_bwd   per-head RMS norm and rotation of queries and keys, laid out for
                   attn_fwd, and its gradients
  append           the same pass writing K and V into the paged bf16 cache
  append4          the same pass writing K and V into the paged 4-bit cache, then the
                   cached history read back
  decode4          one query token per request against the 4-bit cache
  prefill4         a chunk of new tokens per request against the 4-bit cache

The 4-bit cache.  A pool is uint8 [blocks, Hkv, 18 D]: for each (block of 16 tokens, KV
head) the K codes (16 rows of D / 2 bytes), the K scales (16 rows of D / 32 bf16), then
the same for V.  32 channels of one token share a scale s: the largest magnitude / 7,
rounded to 5 significant bits.  A channel is n = round(x / s) in [-7, 7], held as n + 8.
The nibbles of a K row run over (c % 32) / 8, then c / 32, then c % 8 (slowest first),
those of a V row over (c % 32) / 4, c / 32, c % 4; the low nibble of a byte comes first.
"""

import math
import random

import torch

own = False

BS = 16  # tokens in a block of the paged cache


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # a long prompt of a grouped-query model, packed projection rows, all of it new
        dict(name="rope_prompt_16k", kind="rope", B=1, T=16384, Hq=32, Hkv=8, D=128, rot=128,
             norm=True, interleaved=False, start=0),
        # a small odd batch: partial interleaved rotation, no norm, positions behind a prefix
        dict(name="rope_odd_d64", kind="rope", B=3, T=777, Hq=12, Hkv=2, D=64, rot=32,
             norm=False, interleaved=True, start=1000),
        # a training step of the 4 x 2048 multi-head workload
        dict(name="rope_bwd_mha_2k", kind="rope_bwd", B=4, T=2048, Hq=16, Hkv=16, D=128, rot=128,
             norm=True, interleaved=False, start=0),
        # one new token for each of 64 requests: latency counts
        dict(name="append_64x1", kind="append", S=64, Tn=1, Hq=12, Hkv=2, D=128, rot=128,
             norm=True, interleaved=False, lo=512, hi=2048, lens=5003),
        # a prompt chunk of 16 requests
        dict(name="append_16x512", kind="append", S=16, Tn=512, Hq=32, Hkv=8, D=128, rot=128,
             norm=True, interleaved=False, lo=0, hi=1024, lens=6003),
        # the first generated tokens of 64 short requests over the 4-bit cache
        dict(name="append4_64x1", kind="append4", S=64, Tn=1, Hq=12, Hkv=2, D=128, rot=128,
             norm=True, interleaved=False, lo=0, hi=63, lens=5004),
        # 16 first prompt chunks into the 4-bit cache
        dict(name="append4_16x512", kind="append4", S=16, Tn=512, Hq=32, Hkv=8, D=128, rot=128,
             norm=True, interleaved=False, lo=0, hi=0, lens=6004),
        # the 64-request decode workload
        dict(name="decode4_64req", kind="decode4", S=64, Hq=12, Hkv=2, D=128, lo=512, hi=8192,
             lens=5003),
        # one long conversation
        dict(name="decode4_1x128k", kind="decode4", S=1, Hq=32, Hkv=8, D=128, lo=131000, hi=131000,
             lens=5005),
        # a few short requests, narrow heads, 16 query heads on one KV head
        dict(name="decode4_odd_d64", kind="decode4", S=5, Hq=16, Hkv=1, D=64, lo=1, hi=300,
             lens=5006),
        # chunked prefill: 16 requests x 512 new tokens
        dict(name="prefill4_16x512", kind="prefill4", S=16, Tn=512, Hq=32, Hkv=8, D=128,
             causal=True, lo=1024, hi=8192, lens=6003),
        # a few drafted tokens of three requests to be verified, narrow heads
        dict(name="prefill4_odd_d64", kind="prefill4", S=3, Tn=37, Hq=8, Hkv=2, D=64, causal=True,
             lo=37, hi=500, lens=6005),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_bwd", "append", "append4", "decode4", "decode4", "prefill4",
                       "prefill4"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    while Hq > 48:
        Hq //= 2
        Hq -= Hq % Hkv
    c = dict(kind=kind, Hq=Hq, Hkv=Hkv, D=D)
    if kind in ("rope", "rope_bwd"):
        T = _log(rng, 1, 8192)
        c |= dict(B=max(1, min(_log(rng, 1, 64), 8192 // T)), T=T, start=rng.randrange(0, 4000))
    elif kind in ("append", "append4"):
        Tn = _log(rng, 1, 700)
        hi = _log(rng, 1, 1000)
        c |= dict(S=max(1, min(_log(rng, 1, 128), 8192 // Tn)), Tn=Tn, lo=0, hi=hi,
                  lens=rng.randrange(1 << 30))
        if kind == "append4" and c["S"] * (hi + Tn) > 20000:
            c["S"] = max(1, 20000 // (hi + Tn))
    elif kind == "decode4":
        hi = _log(rng, 1, 60000)
        c |= dict(S=max(1, min(_log(rng, 1, 200), 1000000 // (hi * Hkv))),
                  lo=min(hi, rng.choice([0, 1, 100])),
                  hi=hi, lens=rng.randrange(1 << 30))
    else:
        Tn = _log(rng, 1, 900)
        hi = Tn + _log(rng, 1, 6000)
        c |= dict(S=max(1, min(_log(rng, 1, 16), 10 ** 11 // (Tn * hi * Hq * D))), Tn=Tn,
                  causal=rng.random() < 0.8, lo=rng.choice([0, Tn]), hi=hi, lens=rng.randrange(1 << 30))
    if kind in ("rope", "rope_bwd", "append", "append4"):
        c |= dict(rot=rng.choice([D, D, D // 2, 24]), norm=rng.random() < 0.7,
                  interleaved=rng.random() < 0.3)
    return c


def _lens(c):
    """Cached tokens of each request (before the new ones, for the appends)."""
    rng = random.Random(c["lens"])
    return [rng.randint(c["lo"], c["hi"]) for _ in range(c["S"])]


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
EPS = 1e-6
THETA = 1e6


def _table(n, rot):
    """cos | sin of position p times theta^(-2 i / rot), angles in 64 bits."""
    inv = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _quantise(x):
    """Codes n + 8 (uint8, the shape of x) and scales (bf16, [..., D / 32]) of bf16 rows."""
    g = x.float().unflatten(-1, (-1, 32))
    t = g.abs().amax(-1) / 7.0
    b = t.view(torch.int32)
    b = (b + 0x3FFFF + ((b >> 19) & 1)) & ~0x7FFFF
    s = torch.where(t.isfinite(), b.view(torch.float32), torch.nan)
    d = torch.where((s > 0) & s.isfinite(), s, 1.0)
    n = torch.where((s > 0)[..., None], g / d[..., None], 0.0).round().clamp(-7, 7)
    return (n + 8).to(torch.uint8).flatten(-2), s.bfloat16()


def _pack(n, per):
    """Codes of rows [..., D] -> bytes [..., D / 2]; per = 8 for K rows, 4 for V rows."""
    n = n.unflatten(-1, (-1, 32 // per, per)).transpose(-3, -2).flatten(-3)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpack(b, per):
    """Bytes [..., D / 2] -> codes [..., D]."""
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return n.unflatten(-1, (32 // per, -1, per)).transpose(-3, -2).flatten(-3)


def _pool_parts(pool):
    """Views of a pool: K codes, K scales, V codes, V scales, each [blocks, Hkv, 16, .]."""
    D = pool.shape[2] // 18
    cut = pool.split([8 * D, D, 8 * D, D], 2)
    return [t.unflatten(2, (BS, -1)) for t in cut]


def _paged(c, lens, gen, four):
    """Block table (a random permutation of the pool) and pools of used and spare blocks."""
    S, Hkv, D = c["S"], c["Hkv"], c["D"]
    blocks = torch.tensor([-(-n // BS) for n in lens])
    used = int(blocks.sum())
    NB = max(1, used + -(-used // 8))
    perm = torch.randperm(NB, generator=gen, device="cuda").int()
    mb = max(1, int(blocks.max()))
    col = torch.arange(mb)[None, :]
    index = (blocks.cumsum(0) - blocks)[:, None] + col
    live = (col < blocks[:, None]).cuda()
    table = torch.where(live, perm[index.clamp(max=NB - 1).cuda()], -1)
    gain = torch.exp(0.3 * torch.randn(2, Hkv, 1, D, generator=gen, device="cuda"))
    k = (torch.randn(NB, Hkv, BS, D, generator=gen, device="cuda") * gain[0]).bfloat16()
    v = (torch.randn(NB, Hkv, BS, D, generator=gen, device="cuda") * gain[1]).bfloat16()
    if not four:
        return table, k, v
    pool = torch.empty(NB, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    parts = _pool_parts(pool)
    for x, codes, scales, per in ((k, parts[0], parts[1], 8), (v, parts[2], parts[3], 4)):
        n, s = _quantise(x)
        codes.copy_(_pack(n, per))
        scales.copy_(s.view(torch.uint8))
    return table, pool


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    st = dict(c)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["kind"] in ("rope", "rope_bwd", "append", "append4"):
        B, T = (c["B"], c["T"]) if "B" in c else (c["S"], c["Tn"])
        # the rows a fused projection puts out, with channels of unlike size
        rows = randn(B, T, Hq + 2 * Hkv, D) * torch.exp(0.3 * randn(Hq + 2 * Hkv, D))
        st["q"], st["k"], st["v"] = rows.bfloat16().split([Hq, Hkv, Hkv], 2)
        st["wq"] = (1 + 0.1 * randn(D)).bfloat16() if c["norm"] else None
        st["wk"] = (1 + 0.1 * randn(D)).bfloat16() if c["norm"] else None
        if "B" in c:
            st["cs"] = _table(c["start"] + B + T, c["rot"])
            first = c["start"] + torch.arange(B, device="cuda")[:, None]
            st["pos"] = (first + torch.arange(T, device="cuda")).int()
        else:
            st["cs"] = _table(c["hi"] + T, c["rot"])
    if c["kind"] == "rope_bwd":
        st["gq"], st["gk"], st["gv"] = (randn(c["B"], h, c["T"], D).bfloat16() for h in (Hq, Hkv, Hkv))
    if "S" in c:
        lens = _lens(c)
        after = [n + c["Tn"] for n in lens] if c["kind"].startswith("append") else lens
        st["max_len"] = max(1, max(after))
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["new"] = torch.empty_like(st["lens"])
        if c["kind"] == "append":
            st["table"], st["kp"], st["vp"] = _paged(c, after, gen, False)
        else:
            st["table"], st["pool"] = _paged(c, after, gen, True)
        if c["kind"] == "append4":
            st["hk"], st["hv"] = (torch.zeros(c["S"], Hkv, st["max_len"], D, dtype=torch.bfloat16,
                                              device="cuda") for _ in range(2))
        if c["kind"] == "decode4":
            st["q"] = randn(c["S"], Hq, D).bfloat16()
        if c["kind"] == "prefill4":
            st["q"] = randn(c["S"], Hq, c["Tn"], D).bfloat16()
    return st


# --------------------------------------------------------------------------- #
# the plain form
# --------------------------------------------------------------------------- #
def _rotate(x, cs, rot, interleaved, back=False):
    """The first `rot` channels of fp32 rows [B, T, H, D], by rows [B, T, rot] of the table."""
    cos, sin = cs[:, :, None].chunk(2, -1)
    if back:
        sin = -sin
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, rest], -1)


def _norm_rope(x, w, cs, st):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(x, cs, st["rot"], st["interleaved"]).bfloat16()


def _norm_rope_bwd(g, x, w, cs, st):
    g = _rotate(g.transpose(1, 2).float(), cs, st["rot"], st["interleaved"], back=True)
    if w is None:
        return g.bfloat16(), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dw = (g * xh).sum((0, 1, 2), dtype=torch.float64).float()
    g = g * w.float()
    return (r * (g - xh * (g * xh).mean(-1, keepdim=True))).bfloat16(), dw


def _slots(st, Tn):
    """Physical block and slot [S, Tn] of each request's new tokens, and their positions."""
    pos = st["lens"].long()[:, None] + torch.arange(Tn, device="cuda")
    return st["table"].long().gather(1, pos // BS), pos % BS, pos


def _values(codes, scales, per):
    n = _unpack(codes, per).float() - 8
    s = scales.contiguous().view(torch.bfloat16).float()
    return (n.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _history(st, lens):
    """K and V of every request in logical order, fp32 [S, Hkv, L, D], zero past its length."""
    L = st["max_len"]
    t = torch.arange(L, device="cuda")
    blk, live = st["table"].long()[:, t // BS].clamp(min=0), t < lens[:, None]
    kc, ks, vc, vs = (p[blk, :, t % BS] for p in _pool_parts(st["pool"]))  # [S, L, Hkv, .]
    live = live[:, None, :, None]
    return (torch.where(live, _values(a, s, per).transpose(1, 2), 0.0)
            for a, s, per in ((kc, ks, 8), (vc, vs, 4)))


def _attend(q, k, v, mask, scale):
    """softmax(scale q k^T) v with the heads of one KV head as rows: q [S, Hkv, R, D] and
    mask [S, R, L]; a row whose mask leaves nothing gives 0 and -inf."""
    s = (q.float() @ k.transpose(2, 3)) * scale
    s = s.masked_fill_(~mask[:, None], -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(torch.where(m.isfinite(), m, 0.0)))
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l > 0, l, 1.0)
    return o.bfloat16(), (m + torch.log(l)).squeeze(-1)


def _plain(st):
    kind = st["kind"]
    if kind in ("rope", "rope_bwd"):
        cs = st["cs"][st["pos"].long()]
        if kind == "rope":
            y = [_norm_rope(st["q"], st["wq"], cs, st), _norm_rope(st["k"], st["wk"], cs, st),
                 st["v"]]
            return [t.transpose(1, 2).contiguous() for t in y]
        dq, dwq = _norm_rope_bwd(st["gq"], st["q"], st["wq"], cs, st)
        dk, dwk = _norm_rope_bwd(st["gk"], st["k"], st["wk"], cs, st)
        return [dq, dk, st["gv"].transpose(1, 2).contiguous(), dwq, dwk]
    if kind in ("append", "append4"):
        blk, slot, pos = _slots(st, st["Tn"])
        cs = st["cs"][pos]
        q = _norm_rope(st["q"], st["wq"], cs, st).transpose(1, 2).contiguous()
        k = _norm_rope(st["k"], st["wk"], cs, st)
        st["new"].copy_(st["lens"] + st["Tn"])
        if kind == "append":
            st["kp"][blk, :, slot] = k
            st["vp"][blk, :, slot] = st["v"]
            return [q, st["new"], st["kp"], st["vp"]]
        kc, ks, vc, vs = _pool_parts(st["pool"])
        (nk, sk), (nv, sv) = _quantise(k), _quantise(st["v"])
        kc[blk, :, slot], vc[blk, :, slot] = _pack(nk, 8), _pack(nv, 4)
        ks[blk, :, slot], vs[blk, :, slot] = sk.view(torch.uint8), sv.view(torch.uint8)
        hk, hv = _history(st, st["new"])
        return [q, st["new"], st["hk"].copy_(hk), st["hv"].copy_(hv)]
    # attention
    S, Hq, Hkv, D = st["S"], st["Hq"], st["Hkv"], st["D"]
    Tn = st.get("Tn", 1)
    k, v = _history(st, st["lens"])
    end = st["lens"].long()[:, None]
    if st.get("causal"):
        end = end - Tn + 1 + torch.arange(Tn, device="cuda")
    mask = torch.arange(st["max_len"], device="cuda") < end[..., None]  # [S, 1 or Tn, L]
    mask = mask.expand(S, Tn, -1).repeat(1, Hq // Hkv, 1)
    o, lse = _attend(st["q"].reshape(S, Hkv, -1, D), k, v, mask, 1 / math.sqrt(D))
    return [o.reshape(st["q"].shape), lse.reshape(st["q"].shape[:-1])]


# --------------------------------------------------------------------------- #
# the library's calls
# --------------------------------------------------------------------------- #
def _calls(st):
    import attention_flashattention_fwd_03_gb300 as gb

    kind = st["kind"]
    if kind in ("decode4", "prefill4"):
        attend = gb.paged_kv4_attn_decode if kind == "decode4" else gb.paged_kv4_attn_prefill
        how = {} if kind == "decode4" else {"causal": st["causal"]}
        return list(attend(st["q"], st["pool"], st["table"], st["lens"], st["max_len"], **how))
    how = dict(cos_sin=st["cs"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
               interleaved=st["interleaved"])
    if kind == "rope":
        return list(gb.qkv_norm_rope(st["q"], st["k"], st["v"], positions=st["pos"], **how))
    if kind == "rope_bwd":
        return list(gb.qkv_norm_rope_bwd(st["gq"], st["gk"], st["gv"], st["q"], st["k"],
                                         positions=st["pos"], **how))
    if kind == "append":
        q, new = gb.paged_qkv_append(st["q"], st["k"], st["v"], st["kp"], st["vp"], st["table"],
                                     st["lens"], new_seq_lens=st["new"], **how)
        return [q, new, st["kp"], st["vp"]]
    q, new = gb.paged_kv4_append(st["q"], st["k"], st["v"], st["pool"], st["table"], st["lens"],
                                 new_seq_lens=st["new"], **how)
    hk, hv = gb.paged_kv4_gather(st["pool"], st["table"], new, st["max_len"], k_out=st["hk"],
                                 v_out=st["hv"])
    return [q, new, hk, hv]


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    row4 = 9 * D // 8  # bytes of K and V of one token and KV head: 2 x (D / 2 + D / 16)
    if c["kind"] in ("rope", "rope_bwd"):
        n = c["B"] * c["T"]
        rows = n * (Hq + 2 * Hkv) * D * 2
        extra = n * 4 + min(n, c["T"] + c["B"]) * c["rot"] * 4
        if c["kind"] == "rope":
            return {"bytes": 2 * rows + extra, "flops": 8 * n * (Hq + Hkv) * D}
        x = n * (Hq + Hkv) * D * 2 if c["norm"] else 0
        return {"bytes": 2 * rows + x + extra, "flops": 16 * n * (Hq + Hkv) * D}
    lens = _lens(c)
    total, S = sum(lens), c["S"]
    if c["kind"] in ("append", "append4"):
        n = S * c["Tn"]
        q, kv = n * Hq * D * 2, n * Hkv * D * 4
        extra = min(n, c["hi"] + c["Tn"]) * c["rot"] * 4 + 8 * S
        flops = 8 * n * (Hq + 2 * Hkv) * D
        if c["kind"] == "append":
            return {"bytes": 2 * q + 2 * kv + extra, "flops": flops}
        history = (total + n) * Hkv * (row4 + 4 * D)
        return {"bytes": 2 * q + kv + n * Hkv * row4 + history + extra, "flops": flops}
    Tn = c.get("Tn", 1)
    rows = S * Tn * Hq
    if c.get("causal"):
        pairs = sum(max(0, L - i) for L in lens for i in range(Tn))
    else:
        pairs = total * Tn
    return {"bytes": rows * (4 * D + 4) + total * Hkv * row4 + S * 4 + total // BS * 4,
            "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def _exact_rows(x, w, cs, c):
    """Norm and rotation channel by channel; x [B, T, H, D] fp64, cs [B, T, rot] fp64."""
    if w is not None:
        x = w.double() * x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / x.shape[-1] + EPS)
    half = c["rot"] // 2
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    y = x.clone()
    co, si = cs[:, :, None, :half], cs[:, :, None, half:]
    y[..., a] = co * x[..., a] - si * x[..., b]
    y[..., b] = si * x[..., a] + co * x[..., b]
    return y


def _exact_values(x):
    """What the 4-bit cache holds for bf16 rows [..., D], in 64 bits."""
    g = x.double().reshape(*x.shape[:-1], -1, 32)
    man, ex = torch.frexp(g.abs().amax(-1) / 7)  # man in [1/2, 1)
    s = torch.ldexp(torch.round(man * 32) / 32, ex)[..., None]
    n = torch.where(s > 0, torch.clamp(torch.round(g / s), -7, 7), 0.0)
    return (n * s).reshape(x.shape)


def _exact_cached(pool, table, r, n):
    """K and V [Hkv, n, D] fp64 of request r, read nibble by nibble."""
    D = pool.shape[2] // 18
    t = torch.arange(n, device="cuda")
    c = torch.arange(D, device="cuda")
    rows = pool[table[r].long()[t // BS]]  # [n, Hkv, 18 D]
    out = []
    for base, per in ((0, 8), (9 * D, 4)):
        nib = ((c % 32) // per * (D // 32) + c // 32) * per + c % per
        at = (base + (t % BS)[:, None] * (D // 2) + nib // 2)[:, None].expand(n, rows.shape[1], D)
        code = (rows.gather(2, at).long() >> (4 * (nib % 2))) & 15
        at = base + 8 * D + (t % BS)[:, None] * (D // 16) + c // 32 * 2
        lo, hi = (rows.gather(2, (at + i)[:, None].expand(n, rows.shape[1], D)).int() for i in (0, 1))
        s = ((lo << 16) | (hi << 24)).view(torch.float32).double()
        out.append(((code - 8) * s).transpose(0, 1))
    return out


def exact(case, seed):
    c, st = case, prepare(case, seed)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["kind"] == "rope":
        cs = st["cs"].double()[st["pos"].long()]
        q, k = (_exact_rows(st[x].double(), st["w" + x], cs, c) for x in "qk")
        return [x.permute(0, 2, 1, 3) for x in (q, k, st["v"].double())]
    if c["kind"] == "rope_bwd":
        cs = st["cs"].double()[st["pos"].long()]
        out, dws = [], []
        for x in "qk":  # the gradient of sum(g * y), by differentiation
            leaf = st[x].double().requires_grad_()
            w = st["w" + x].double().requires_grad_() if c["norm"] else None
            y = _exact_rows(leaf, w, cs, c)
            got = torch.autograd.grad((y * st["g" + x].double().permute(0, 2, 1, 3)).sum(),
                                      [leaf] + ([w] if c["norm"] else []))
            out.append(got[0])
            dws.append(got[1] if c["norm"] else None)
        return out + [st["gv"].double().permute(0, 2, 1, 3)] + dws
    lens = st["lens"].tolist()
    if c["kind"] in ("append", "append4"):
        pos = st["lens"].long()[:, None] + torch.arange(c["Tn"], device="cuda")
        cs = st["cs"].double()[pos]
        q, k = (_exact_rows(st[x].double(), st["w" + x], cs, c) for x in "qk")
        v, q = st["v"].double(), q.permute(0, 2, 1, 3)
        new = st["lens"] + c["Tn"]
        if c["kind"] == "append":
            kp, vp = st["kp"].double(), st["vp"].double()
            for r, n in enumerate(lens):
                at = torch.arange(n, n + c["Tn"], device="cuda")
                kp[st["table"][r].long()[at // BS], :, at % BS] = k[r]
                vp[st["table"][r].long()[at // BS], :, at % BS] = v[r]
            return [q, new, kp, vp]
        hk, hv = (torch.zeros(c["S"], Hkv, st["max_len"], D, dtype=torch.float64, device="cuda")
                  for _ in range(2))
        k, v = _exact_values(k.bfloat16()).permute(0, 2, 1, 3), _exact_values(v).permute(0, 2, 1, 3)
        for r, n in enumerate(lens):
            hk[r, :, :n], hv[r, :, :n] = _exact_cached(st["pool"], st["table"], r, n)
            hk[r, :, n:n + c["Tn"]], hv[r, :, n:n + c["Tn"]] = k[r], v[r]
        return [q, new, hk, hv]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:-1], -torch.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        if n == 0:
            continue
        k, v = _exact_cached(st["pool"], st["table"], r, n)
        for h in range(Hq):
            s = st["q"][r, h].double().reshape(-1, D) @ k[h // (Hq // Hkv)].T / math.sqrt(D)
            if c.get("causal"):
                i = torch.arange(c["Tn"], device="cuda")[:, None]
                s[torch.arange(n, device="cuda") > n - c["Tn"] + i] = -torch.inf
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.where(z.isfinite(), torch.exp(s - torch.where(z.isfinite(), z, 0.0)), 0.0)
            o[r, h] = (p @ v[h // (Hq // Hkv)]).reshape(o[r, h].shape)
            lse[r, h] = z.reshape(lse[r, h].shape)
    return [o, lse]
