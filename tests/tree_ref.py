"""Plain 64-bit implementations of the operators for trees of drafted tokens, and inputs for
their tests (test infrastructure only)."""

from __future__ import annotations

from fractions import Fraction

import numpy as np

import oracle
import synth


def ancestors(parents, n):
    """[n, n]: whether node j is node i or an ancestor of it."""
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        a = i
        while a >= 0:
            seen[i, a] = True
            a = int(parents[a])
    return seen


def tree(kind, Tn, rng):
    """Parents of a tree: a chain, a star of roots, a binary tree, or at random."""
    i = np.arange(Tn)
    if kind == "chain":
        return i - 1
    if kind == "star":
        return np.full(Tn, -1)
    if kind == "binary":
        return (i - 1) // 2 if Tn else i
    if kind == "comb":  # a chain with a leaf at each of its nodes
        return np.where(i % 2 == 0, i - 2, i - 1).clip(-1)
    p = np.floor(i * rng.random(Tn) ** 1.5).astype(int)
    return np.where(rng.random(Tn) < 0.1, -1, np.minimum(p, i - 1))


def attention(q, k_pool, v_pool, table, lens, parents, nodes, scale):
    """O, LSE, the mean magnitude sum p |v|, and a bound on the rounding of a score in fp32, all
    float64, for bf16 bits."""
    S, Hq, Tn, D = q.shape
    Hkv = k_pool.shape[1]
    f = lambda b: synth.bf16_bits_to_float(b).astype(np.float64)  # noqa: E731
    o = np.zeros((S, Hq, Tn, D))
    mag = np.zeros((S, Hq, Tn, D))
    lse = np.full((S, Hq, Tn), -np.inf)
    dev = np.zeros((S, Hq, Tn))
    for r in range(S):
        L, n = int(lens[r]), int(nodes[r])
        if n == 0:
            continue
        mask = np.concatenate([np.ones((n, L), bool), ancestors(parents[r], n)], 1)
        both = np.array([L + n], dtype=np.int32)
        for h in range(Hkv):
            k = f(oracle.paged_gather(k_pool, table[r:r + 1], both, 0, h))
            v = f(oracle.paged_gather(v_pool, table[r:r + 1], both, 0, h))
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = f(q[r, g, :n])
                s = np.where(mask, x @ k.T * scale, -np.inf)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(1, keepdims=True)
                lse[r, g, :n] = (m + np.log(z))[:, 0]
                o[r, g, :n] = e / z @ v
                mag[r, g, :n] = e / z @ np.abs(v)
                # D products and sums of fp32, each off by 2^-23 of the sum of magnitudes at most
                dev[r, g, :n] = (np.abs(x) @ np.abs(k).T * scale * D * 2.0 ** -23).max(1)
    return o, lse, mag, dev


def check_attention(got_o, got_lse, ref, nodes, keys, rows=None):
    """What may differ: probabilities rounded to bf16 (2^-8 of the magnitude), the result
    rounded to bf16 (2^-8 of it), scores by `dev` each (which moves a probability and the sum by
    e^dev - 1 <= 2 dev), exp2 by 2^-20, and sums of `keys` terms in fp32, truncated perhaps (2^-23
    each)."""
    o, lse, mag, dev = ref
    delta = (4 * dev + 2.0 ** -19 + 2 * keys * 2.0 ** -23)[..., None]
    tol = 2.0 ** -8 * (1 + 2.0 ** -8) * mag + 2.0 ** -8 * np.abs(o) + delta * mag + 2.0 ** -126
    fin = np.where(np.isfinite(lse), np.abs(lse), 0)
    ltol = 2 * dev + 2.0 ** -20 + keys * 2.0 ** -23 + 2.0 ** -22 * fin
    for r in range(o.shape[0]) if rows is None else rows:
        n = int(nodes[r])
        assert np.all(got_o[r, :, n:] == 0) and np.all(np.isneginf(got_lse[r, :, n:])), r
        assert np.all(np.isfinite(got_o[r])), r
        assert np.all(np.abs(got_o[r] - o[r]) <= tol[r]), (r, np.abs(got_o[r] - o[r]).max())
        assert np.all(np.abs(got_lse[r, :, :n] - lse[r, :, :n]) <= ltol[r, :, :n]), r


class TreeInputs:
    """Pools, table, queries and trees; every slot outside a request's tokens and nodes is NaN."""

    def __init__(self, Hq, Hkv, D, Tn, lens, kind="random", nodes=None, seed=70000, slack=0):
        rng = np.random.default_rng(seed)
        S = len(lens)
        self.nodes = np.full(S, Tn) if nodes is None else np.array(nodes)
        self.lens = np.array(lens, dtype=np.int32)
        keys = self.lens + self.nodes
        cfg = synth.DecodeConfig("tree", S, Hq, Hkv, D, 0, 1, 16, seed)
        self.max_len = int(max(keys.max(), 1)) + slack
        p = synth.paged_inputs(cfg, seq_lens=keys.tolist(), max_seq_len=self.max_len)
        self.k_pool, self.v_pool, self.table = p.k_pool, p.v_pool, p.block_table
        self.scale = cfg.softmax_scale
        self.q = synth.normal_bf16(seed + 11, (S, Hq, Tn, D))
        self.parents = np.stack([tree(kind, Tn, rng) for _ in range(S)]).astype(np.int32).reshape(S, Tn)
        self.ragged = nodes is not None

    def ref(self):
        return attention(self.q, self.k_pool, self.v_pool, self.table, self.lens, self.parents,
                         self.nodes, self.scale)

    @property
    def keys(self):
        return (self.lens + self.nodes)[:, None, None].astype(np.float64)


def verify_exact(p, q, tokens, parents, u, n, V):
    """One request in rational numbers: (tokens put out, nodes that stand).  p and q are lists
    of rows of numbers that Fraction takes."""
    if n == 0:
        return [], []
    cur, path, out = 0, [0], []
    w, W = [Fraction(x) for x in p[0]], Fraction(1)
    for i in range(1, n):
        if parents[i] != cur:
            continue
        x = int(tokens[i])
        inside = 0 <= x < V
        if q is None:
            row = [Fraction(1 if y == x else 0) for y in range(V)]
            qx = Fraction(1)
        else:
            row = [Fraction(y) for y in q[cur]]
            qx = row[x] if inside else Fraction(0)
        if Fraction(u[i]) * qx * W < (w[x] if inside else 0):
            cur = i
            path.append(i)
            out.append(x)
            w, W = [Fraction(y) for y in p[i]], Fraction(1)
            continue
        rest = [max(a - W * b, Fraction(0)) for a, b in zip(w, row)]
        if sum(rest) > 0:
            w, W = rest, sum(rest)
    total, run, last = sum(w), Fraction(0), -1
    for y in range(V):
        run += w[y]
        if run > Fraction(u[0]) * total:
            last = y
            break
    return out + [last], path


def verify_plain(p, q, tokens, parents, u, n):
    """The same in float64, for longer rows."""
    if n == 0:
        return [], []
    cur, path, out = 0, [0], []
    w, W = p[0].astype(np.float64), 1.0
    for i in range(1, n):
        if parents[i] != cur:
            continue
        x = int(tokens[i])
        if q is None:
            row = np.zeros_like(w)
            row[x] = 1
        else:
            row = q[cur].astype(np.float64)
        if float(u[i]) * row[x] * W < w[x]:
            cur = i
            path.append(i)
            out.append(x)
            w, W = p[i].astype(np.float64), 1.0
            continue
        rest = np.maximum(w - W * row, 0)
        if rest.sum() > 0:
            w, W = rest, rest.sum()
    c = np.cumsum(w)
    last = int(np.searchsorted(c, float(u[0]) * c[-1], side="right"))
    return out + [last if last < len(w) else -1], path


def keep(pool, table, lens, path, counts):
    """A pool [blocks, Hkv, 16, D] after the kept rows have been moved together."""
    out = pool.copy()
    for r, L in enumerate(lens):
        rows = [pool[table[r, (L + i) // 16], :, (L + i) % 16].copy() for i in path[r][:counts[r]]]
        for j, row in enumerate(rows):
            out[table[r, (L + j) // 16], :, (L + j) % 16] = row
    return out
